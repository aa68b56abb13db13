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
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 bf16x4_u __attribute__((ext_vector_type(4), aligned(2)));

struct Args {
    const int8_t* x;
    const float* xs;
    const int8_t* w;
    const float* ws;
    void* y;
    int32_t M, N, Kin;
};

// Four outputs of a row, `left` of them (at least one) inside it.  Rows start
// on any 4 bytes (bf16: 2): one store of 16 (8) bytes needs no more than that.
template <int YT>
__device__ __forceinline__ void store_quad(void* y, int64_t at, const float (&v)[4], int left)
{
    if (left >= 4) {
        if (YT == TQ_F32) *(f32x4_u*)((float*)y + at) = f32x4_u{v[0], v[1], v[2], v[3]};
        else *(bf16x4_u*)((__bf16*)y + at) = bf16x4_u{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (e < left) {
            if (YT == TQ_F32) ((float*)y)[at + e] = v[e];
            else ((__bf16*)y)[at + e] = (__bf16)v[e];
        }
}

// ---------------------------------------------------------------------------
// Few tokens: the weight is read once, straight into MFMA operands.  A wave
// owns 16 RT rows of w and 16 MT tokens; W waves split the columns, 128 at a
// time in turn, and add their sums in LDS (integers: any order).  G such
// groups make a workgroup.  A unit of 128 columns is a whole line of each row
// (two MFMA steps); D units per wave are in flight.  Loads go through buffer
// resources: lanes past M, N or Kin read zeros without touching memory.
template <int YT, int MT, int RT, int W, int G, int D>
__global__ __launch_bounds__(64 * W * G) void k_dense_i8_few(Args A, int blocks_m)
{
    __shared__ i32x4 red[W > 1 ? G : 1][W > 1 ? W : 1][W > 1 ? RT * MT : 1][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
    const int g = wave / W, part = wave % W;
    const int m0 = (int)(blockIdx.x % blocks_m) * 16 * MT, n0 = ((int)(blockIdx.x / blocks_m) * G + g) * 16 * RT;
    const int K = A.Kin, U = (K + 127) >> 7;
    const int mrows = A.M - m0 < 16 * MT ? A.M - m0 : 16 * MT;
    const int nrows = n0 >= A.N ? 0 : A.N - n0 < 16 * RT ? A.N - n0 : 16 * RT;
    const __amdgpu_buffer_rsrc_t rx = rsrc(A.x + (int64_t)m0 * K, (int64_t)mrows * K);
    const __amdgpu_buffer_rsrc_t rw = rsrc(A.w + (int64_t)(nrows ? n0 : 0) * K, (int64_t)nrows * K);
    uint32_t xo[MT], wo[RT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xo[m] = 16 * m + r < mrows ? (uint32_t)(16 * m + r) * (uint32_t)K + 16 * q : kOffNone;
#pragma unroll
    for (int n = 0; n < RT; ++n) wo[n] = 16 * n + r < nrows ? (uint32_t)(16 * n + r) * (uint32_t)K + 16 * q : kOffNone;
    i32x4 acc[RT][MT];
#pragma unroll
    for (int n = 0; n < RT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = i32x4{0, 0, 0, 0};
    u32x4 fx[D][2][MT], fw[D][2][RT];
    auto load = [&](int d, int u) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int col = u * 128 + h * 64;
            const bool in = col + 16 * q < K;             // also false past the last unit
#pragma unroll
            for (int n = 0; n < RT; ++n)
                fw[d][h][n] = buffer_load<u32x4, 0>(rw, in ? wo[n] + col : kOffNone, 0);
#pragma unroll
            for (int m = 0; m < MT; ++m) fx[d][h][m] = buffer_load<u32x4, 0>(rx, in ? xo[m] + col : kOffNone, 0);
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, part + d * W);
    for (int u = part; u < U; u += D * W) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < RT; ++n)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[n][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, fw[d][h][n]),
                                                                          __builtin_bit_cast(i32x4, fx[d][h][m]),
                                                                          acc[n][m], 0, 0, 0);
            load(d, u + (d + D) * W);
        }
    }
    // lane l holds rows 4 (l / 16) + e of w and token l % 16 of each tile
    auto store = [&](int t, i32x4 v) __attribute__((always_inline)) {
        const int mm = m0 + 16 * (t % MT) + r, nn = n0 + 16 * (t / MT) + 4 * q;
        if (mm >= A.M || nn >= A.N) return;
        const float xs = A.xs[mm];
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = (float)v[e] * (xs * A.ws[nn + e < A.N ? nn + e : A.N - 1]);
        store_quad<YT>(A.y, (int64_t)mm * A.N + nn, f, A.N - nn);
    };
    if constexpr (W == 1) {
#pragma unroll
        for (int t = 0; t < RT * MT; ++t) store(t, acc[t / MT][t % MT]);
    } else {
#pragma unroll
        for (int t = 0; t < RT * MT; ++t) red[g][part][t][lane] = acc[t / MT][t % MT];
        __syncthreads();
        for (int t = part; t < RT * MT; t += W) {
            i32x4 v = red[g][0][t][lane];
#pragma unroll
            for (int p = 1; p < W; ++p) v += red[g][p][t][lane];
            store(t, v);
        }
    }
}

// ---------------------------------------------------------------------------
// Tiles through LDS: a workgroup of 4 waves (2 x 2) owns 32 FM tokens by 32 FN
// rows of w, a wave FM x FN tiles of 16 x 16.
//
// A stage is 128 columns (two MFMA steps) of the tile's rows, row-major with
// 128-byte rows; the 16-byte chunk c of row R sits at slot c ^ (R % 8), so
// that the 8 lanes of one LDS pass (rows R .. R + 7 of one chunk) fall in
// distinct banks.  Loads go from memory straight to LDS: a wave's load fills
// 1 KiB in lane order (8 rows), so the swizzle is applied to the address that
// each lane reads.  Two stages alternate; while the matrix cores run on one
// step's fragments those of the next are read from LDS.  At the second step
// of a stage the waves meet: the next stage has then arrived, and every
// fragment of this one is in registers, so its place takes the loads of the
// stage after the next, spread over the step's MFMAs.
// The first two stages are the last Kin % 256 columns (a whole 256 where that
// is 0), their x fragments past Kin set to zero, so that the loop needs no
// masks.  Rows past M and N are read as the last row (their outputs are not
// stored).
typedef __attribute__((address_space(3))) uint8_t lds_u8;

__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, lds_u8* dst, uint32_t voff, uint32_t soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, voff, soff, 0, 0);
}

// Wait until at most N of this wave's vector memory operations are pending.
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N < 64, "vmcnt field");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);   // lgkmcnt and expcnt at their maxima
}

// One MFMA into accumulators that stay in AGPRs in place.  As a builtin, with
// 256 of them the register allocator moves accumulators between the two
// register files in the loop (about one move per MFMA).  The s_nop covers a
// vector instruction that wrote an operand just before (two wait states).
__device__ __forceinline__ void mfma(i32x4& c, i32x4 a, i32x4 b)
{
    asm volatile("s_nop 1\n\tv_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// Workgroups are dealt to the 8 XCDs in turn: each XCD takes a run of the
// tiles, in strips of kStrip tiles of tokens walked column by column, so that
// its 32 concurrent tiles share few rows of x and w in its L2 (2048 x 6912 x
// 2560: 44.2 -> 41.5 us; strips of 2 or 8 measured alike).
constexpr int kStrip = 4;
__device__ __forceinline__ void tile_of(int id, int tiles_m, int tiles_n, int* tm, int* tn)
{
    const int total = tiles_m * tiles_n, per = total >> 3, rem = total & 7, xcd = id & 7;
    const int s = xcd * per + (xcd < rem ? xcd : rem) + (id >> 3);
    const int strip = s / (kStrip * tiles_n), left = tiles_m - strip * kStrip, wide = left < kStrip ? left : kStrip;
    const int in = s - strip * kStrip * tiles_n;
    *tm = strip * kStrip + in % wide;
    *tn = in / wide;
}

template <int YT, int FM, int FN>
__global__ __launch_bounds__(256) void k_dense_i8_tile(Args A, int tiles_m, int tiles_n)
{
    constexpr int TM = 32 * FM, TN = 32 * FN, XL = TM / 32, WL = TN / 32, NL = XL + WL;   // loads per wave and stage
    constexpr int STAGE = (TM + TN) * 128;
    __shared__ __attribute__((aligned(1024))) uint8_t st0[STAGE], st1[STAGE];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
    int tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, &tm, &tn);
    const int m0 = tm * TM, n0 = tn * TN, K = A.Kin;
    const int mrows = A.M - m0 < TM ? A.M - m0 : TM, nrows = A.N - n0 < TN ? A.N - n0 : TN;
    const __amdgpu_buffer_rsrc_t rx = rsrc(A.x + (int64_t)m0 * K, (int64_t)mrows * K);
    const __amdgpu_buffer_rsrc_t rw = rsrc(A.w + (int64_t)n0 * K, (int64_t)nrows * K);

    // this lane's row in each of the wave's loads (8 rows, 32 apart), and its chunk, the same in all
    const int c = (lane & 7) ^ (lane >> 3);
    uint32_t vo[NL];
#pragma unroll
    for (int l = 0; l < NL; ++l) {
        const int R = ((l < XL ? l : l - XL) * 4 + wave) * 8 + (lane >> 3), rows = l < XL ? mrows : nrows;
        vo[l] = (uint32_t)(R < rows ? R : rows - 1) * (uint32_t)K;
    }
    // the wave's loads l0 .. l1 - 1 of the stage at column `col`; lanes add `off` (their chunk's offset)
    auto request = [&](uint8_t* st, uint32_t col, uint32_t off, int l0, int l1) __attribute__((always_inline)) {
#pragma unroll
        for (int l = l0; l < l1; ++l) {
            const int id = (l < XL ? l : l - XL) * 4 + wave;
            load_lds16(l < XL ? rx : rw, (lds_u8*)st + (l < XL ? 0 : TM * 128) + id * 1024, vo[l] + off, col);
        }
    };
    const int at0 = r * 128 + 16 * (q ^ (r & 7)), at1 = at0 ^ 64;      // chunks q and 4 + q of the lane's row
    const int bx = (wave & 1) * (16 * FM) * 128, bw = TM * 128 + (wave >> 1) * (16 * FN) * 128;
    i32x4 acc[FN][FM];
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int m = 0; m < FM; ++m) acc[n][m] = i32x4{0, 0, 0, 0};
    i32x4 fx0[FM], fw0[FN], fx1[FM], fw1[FN];
    // one step on fragments (x, w); those of the next come from `next` + at.  LOAD: the second step of a stage: the
    // stage at column `col` is requested into `free`, the place of the step's own
    auto step = [&](bool load, i32x4 (&x)[FM], i32x4 (&w)[FN], const uint8_t* next, int at, i32x4 (&xn)[FM],
                    i32x4 (&wn)[FN], uint8_t* free, uint32_t col, uint32_t off) __attribute__((always_inline)) {
        if (load) {
            __builtin_amdgcn_s_waitcnt(0x0070);       // vmcnt(0): the next stage's loads; lgkmcnt(0): this one's reads
            __builtin_amdgcn_s_barrier();
        }
        __builtin_amdgcn_sched_barrier(0);
        // a row of MFMAs covers the reads of one x and one w fragment and, spread, a load or two: all of a step's
        // loads at once hold the wave at their issue while its matrix core idles
#pragma unroll
        for (int n = 0; n < FN; ++n) {
            if (load) request(free, col, off, n * NL / FN, (n + 1) * NL / FN);
            wn[n] = *(const i32x4*)(next + bw + at + n * 2048);
#pragma unroll
            for (int m = n * FM / FN; m < (n + 1) * FM / FN; ++m) xn[m] = *(const i32x4*)(next + bx + at + m * 2048);
#pragma unroll
            for (int m = 0; m < FM; ++m) mfma(acc[n][m], w[n], x[m]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto mask = [&](i32x4 (&x)[FM], int left) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < FM; ++m) x[m] = 16 * q < left ? x[m] : i32x4{0, 0, 0, 0};
    };
    if (K > 0) {
        const int tail = (K & 255) ? K & 255 : 256, main = K - tail;     // the first two stages' columns: main ..
        const int left1 = tail > 128 ? tail - 128 : 0;
        // chunks past Kin are read from the tail's first one
        const uint32_t off = 16 * c, offt0 = 16 * c < tail ? 16 * c : 0, offt1 = 16 * c < left1 ? 128 + 16 * c : 0;
        request(st0, main, offt0, 0, NL);
        request(st1, main, offt1, 0, NL);
        wait_vm<NL>();
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int n = 0; n < FN; ++n) fw0[n] = *(const i32x4*)(st0 + bw + at0 + n * 2048);
#pragma unroll
        for (int m = 0; m < FM; ++m) fx0[m] = *(const i32x4*)(st0 + bx + at0 + m * 2048);
        // the tail's four steps; a stage past the last is requested again from column 0 (or is the tail's own)
        const uint32_t off1 = main > 0 ? off : 0, second = main > 0 ? 128 : 0;
        mask(fx0, tail);
        step(false, fx0, fw0, st0, at1, fx1, fw1, nullptr, 0, 0);
        mask(fx1, tail - 64);
        step(true, fx1, fw1, st1, at0, fx0, fw0, st0, 0, off1);
        mask(fx0, left1);
        step(false, fx0, fw0, st1, at1, fx1, fw1, nullptr, 0, 0);
        mask(fx1, left1 - 64);
        step(true, fx1, fw1, st0, at0, fx0, fw0, st1, second, off1);
        for (int k = 0; k < main; k += 256) {
            const uint32_t next = k + 256 < main ? k + 256 : 0;
            step(false, fx0, fw0, st0, at1, fx1, fw1, nullptr, 0, 0);
            step(true, fx1, fw1, st1, at0, fx0, fw0, st0, next, off);
            step(false, fx0, fw0, st1, at1, fx1, fw1, nullptr, 0, 0);
            step(true, fx1, fw1, st0, at0, fx0, fw0, st1, next + 128, off);
        }
        wait_vm<0>();     // the requests past the last stage: no load may land after the workgroup has left
    }
    // the wait states between the last MFMA and the first read of a result; the reads stay behind it
    asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int m = 0; m < FM; ++m) asm volatile("" : "+a"(acc[n][m]));
    // lane l holds rows 4 (l / 16) + e of w and token l % 16 of each tile
    const int mb = m0 + (wave & 1) * (16 * FM) + r, nb = n0 + (wave >> 1) * (16 * FN) + 4 * q;
    float ws[FN][4], xs[FM];
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) ws[n][e] = A.ws[nb + 16 * n + e < A.N ? nb + 16 * n + e : A.N - 1];
#pragma unroll
    for (int m = 0; m < FM; ++m) xs[m] = A.xs[mb + 16 * m < A.M ? mb + 16 * m : A.M - 1];
    auto store = [&](int m, int n, int left) __attribute__((always_inline)) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)acc[n][m][e] * (xs[m] * ws[n][e]);
        store_quad<YT>(A.y, (int64_t)(mb + 16 * m) * A.N + nb + 16 * n, v, left);
    };
    if (n0 + TN <= A.N) {                                    // tests per four outputs cost 7 us on 4096 x 4096
#pragma unroll
        for (int m = 0; m < FM; ++m)
            if (mb + 16 * m < A.M)
#pragma unroll
                for (int n = 0; n < FN; ++n) store(m, n, 4);
    } else {
#pragma unroll
        for (int n = 0; n < FN; ++n) {
            const int left = A.N - (nb + 16 * n);
            if (left > 0)
#pragma unroll
                for (int m = 0; m < FM; ++m)
                    if (mb + 16 * m < A.M) store(m, n, left);
        }
    }
}

#ifndef FEW_MT1
#define FEW_MT1
#endif

template <int YT, int MT, int RT, int W, int G, int D>
tq_status launch_few_as(const Args& A, hipStream_t st)
{
    const int64_t bm = (A.M + 16 * MT - 1) / (16 * MT), bn = (A.N + 16 * RT * G - 1) / (16 * RT * G);
    if (bm * bn * 64 * W * G > UINT32_MAX)
        return tq_fail(TQ_ERR_UNSUPPORTED, "%lld tiles exceed one launch", (long long)(bm * bn));
    hipLaunchKernelGGL((k_dense_i8_few<YT, MT, RT, W, G, D>), dim3((unsigned)(bm * bn)), dim3(64 * W * G), 0, st, A, (int)bm);
    return TQ_OK;
}

template <int YT, int MT>
tq_status launch_few_m(const Args& A, hipStream_t st)
{
    constexpr int D = MT == 1 ? 4 : MT == 2 ? 3 : 2;
    const int64_t rows = (A.N + 15) / 16;           // 16-row tiles
    if (rows <= 1024) return launch_few_as<YT, MT, 1, 8, 1, D>(A, st);
    if (rows <= 4096) return launch_few_as<YT, MT, 1, 4, 1, D>(A, st);
    return launch_few_as<YT, MT, 1, 2, 2, D>(A, st);
}

template <int YT>
tq_status launch_few(const Args& A, hipStream_t st)
{
    if (A.M <= 16) return launch_few_m<YT, 1>(A, st);
    if (A.M <= 32) return launch_few_m<YT, 2>(A, st);
    return launch_few_m<YT, 4>(A, st);
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
    hipStream_t st = (hipStream_t)stream;
    const auto tiles = [&](int64_t tm, int64_t tn) { return ((M + tm - 1) / tm) * ((N + tn - 1) / tn); };
    if (M > 64) {
        if (tiles(256, 256) > INT32_MAX / 256)
            return tq_fail(TQ_ERR_UNSUPPORTED, "%lld tiles exceed one launch", (long long)tiles(256, 256));
        const int tm = (int)((M + 255) / 256), tn = (int)((N + 32*8-1) / (32*8));
        if (y_type == TQ_F32)
            hipLaunchKernelGGL((k_dense_i8_tile<TQ_F32, 8, 8>), dim3((unsigned)(tm * tn)), dim3(256), 0, st, A, tm, tn);
        else
            hipLaunchKernelGGL((k_dense_i8_tile<TQ_BF16, 8, 8>), dim3((unsigned)(tm * tn)), dim3(256), 0, st, A, tm, tn);
    } else if ((s = y_type == TQ_F32 ? launch_few<TQ_F32>(A, st) : launch_few<TQ_BF16>(A, st))) {
        return s;
    }
    if ((s = tq_check_launch("tq_gemm_dense_i8"))) return s;
    return tq_ok();
}
