// libtq: tq_gemm_dense_i8 -- int8 activations times a dense int8 weight, a
// scale per token and per output channel, on the int8 matrix cores.
//
//   acc[m][n] = sum_i xq[m][i] w[n][i] (int32, exact);
//   y = fl(float(acc) fl(x_scale[m] w_scale[n])).
//
// |acc| <= 128 * 128 * 65536 = 2^30, so int32 never wraps.
#include <math.h>

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
// A few tokens against a narrow weight (M <= 16): too few tiles to fill the
// GPU, so W waves split a 16 x 16 tile's columns, 128 at a time in turn (a
// whole line of each row: two MFMA steps), and add their sums in LDS
// (integers: any order gives the same).  The weight goes from memory straight
// into MFMA operands, two units per wave in flight (four were slower: the
// waves of a compute unit together hold enough); non-temporal loads were 10%
// slower.  Loads go through buffer resources: lanes past M, N or Kin read
// zeros without touching memory.
// 13 x 4096 x 14336: 13.7 us, 4.3 TB/s.
template <int YT, int W>
__global__ __launch_bounds__(64 * W) void k_dense_i8_few(Args A, int tiles_m, int)
{
    constexpr int D = 2;
    __shared__ i32x4 red[W][64];
    const int lane = threadIdx.x & 63, part = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
    const int m0 = (int)(blockIdx.x % tiles_m) * 16, n0 = (int)(blockIdx.x / tiles_m) * 16;
    const int K = A.Kin, U = (K + 127) >> 7;
    const int mrows = A.M - m0 < 16 ? A.M - m0 : 16, nrows = A.N - n0 < 16 ? A.N - n0 : 16;
    const __amdgpu_buffer_rsrc_t rx = rsrc(A.x + (int64_t)m0 * K, (int64_t)mrows * K);
    const __amdgpu_buffer_rsrc_t rw = rsrc(A.w + (int64_t)n0 * K, (int64_t)nrows * K);
    const uint32_t xo = r < mrows ? (uint32_t)r * (uint32_t)K + 16 * q : kOffNone;
    const uint32_t wo = r < nrows ? (uint32_t)r * (uint32_t)K + 16 * q : kOffNone;
    i32x4 acc = {0, 0, 0, 0};
    u32x4 fx[D][2], fw[D][2];
    auto load = [&](int d, int u) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int col = u * 128 + h * 64;
            const bool in = col + 16 * q < K;             // also false past the last unit
            fw[d][h] = buffer_load<u32x4, 0>(rw, in ? wo + col : kOffNone, 0);
            fx[d][h] = buffer_load<u32x4, 0>(rx, in ? xo + col : kOffNone, 0);
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, part + d * W);
    for (int u = part; u < U; u += D * W) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, fw[d][h]),
                                                            __builtin_bit_cast(i32x4, fx[d][h]), acc, 0, 0, 0);
            load(d, u + (d + D) * W);
        }
    }
    red[part][lane] = acc;
    __syncthreads();
    if (part != 0) return;
    // lane l holds rows 4 (l / 16) + e of w and token l % 16
    i32x4 sum = red[0][lane];
#pragma unroll
    for (int p = 1; p < W; ++p) sum += red[p][lane];
    const int m = m0 + r, n = n0 + 4 * q;
    if (m >= A.M || n >= A.N) return;
    const float xs = A.xs[m];
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)sum[e] * (xs * A.ws[n + e < A.N ? n + e : A.N - 1]);
    store_quad<YT>(A.y, (int64_t)m * A.N + n, v, A.N - n);
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
// each lane reads.  While the matrix cores run on one step's fragments those
// of the next are read from LDS.  At the second step of a stage the waves
// meet: the next stage has then arrived, and every fragment of this one is in
// registers, so its place takes the loads of a stage further on, spread over
// the step's MFMAs.
//
// The ring holds NS stages, all of them requested ahead.  The columns are
// walked from the end: the first stage may be short, its x fragments past Kin
// are set to zero, and it starts at the place of the ring from which whole
// turns are left, so that the loop needs no masks and no tests.  KS groups of
// 4 waves share a tile's columns, a block of 128 each in turn, and add their
// sums in LDS.  Rows past M and N are read as the last row (their outputs are
// not stored).
//
// 8192 x 14336 x 4096, bf16 out: 0.41 ms, 2.3 POP/s, the matrix cores busy 54%
// of the time at the clock the power limit leaves (int8 MFMAs alone on random
// values reach 3.2 to 3.9 POP/s, a library product of 8192^3 2.1 POP/s, this
// one 2.6); LDS reads without bank conflicts; what is left over is the
// epilogue, in which all tiles store at once.
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

template <int YT, int FM, int FN, int KS, int NS>
__global__ __launch_bounds__(256 * KS) void k_dense_i8_tile(Args A, int tiles_m, int tiles_n)
{
    constexpr int TM = 32 * FM, TN = 32 * FN, XL = TM / 32, WL = TN / 32, NL = XL + WL;   // loads per wave and stage
    constexpr int STAGE = (TM + TN) * 128;
    static_assert(NS >= 2 && NS <= 4, "stages in the ring");
    // an array per stage: the compiler then sees that a read of one does not wait for the loads into another
    __shared__ __attribute__((aligned(1024))) uint8_t st0_[KS * STAGE], st1_[KS * STAGE],
        st2_[NS > 2 ? KS * STAGE : 16], st3_[NS > 3 ? KS * STAGE : 16];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave_id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = wave_id & 3, group = wave_id >> 2;
    uint8_t* const st0 = st0_ + group * STAGE;
    uint8_t* const st1 = st1_ + group * STAGE;
    uint8_t* const st2 = NS > 2 ? st2_ + group * STAGE : st2_;
    uint8_t* const st3 = NS > 3 ? st3_ + group * STAGE : st3_;
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
        vo[l] = (uint32_t)(R < rows ? R : rows - 1) * (uint32_t)K + 16 * c;
    }
    // Stage j of this group is the block of 128 columns (stages - 1 - j) * KS + group: stage 0 holds the last columns,
    // `valid` of them (none where the block is past Kin)
    const int blocks = (K + 127) >> 7, stages = (blocks + KS - 1) / KS;
    const int last = ((stages - 1) * KS + group) * 128, valid = K - last < 0 ? 0 : K - last < 128 ? K - last : 128;
    // The wave's loads l0 .. l1 - 1 of stage j, lanes moved back by `back`.  Past the last stage loads keep the count:
    // of the tile's first columns, or, with more of them, all of one address.
    auto request = [&](uint8_t* st, int j, uint32_t back, int l0, int l1) __attribute__((always_inline)) {
        const bool live = j < stages;
        const uint32_t col = live ? last - j * KS * 128 : 0;
#pragma unroll
        for (int l = l0; l < l1; ++l) {
            const int id = (l < XL ? l : l - XL) * 4 + wave;
            load_lds16(l < XL ? rx : rw, (lds_u8*)st + (l < XL ? 0 : TM * 128) + id * 1024,
                       NS == 2 || live ? vo[l] - back : 0, col);
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
    // One step: MFMAs on (x, w) while the fragments (xn, wn) are read from `next` + at.  The second step of a stage
    // begins with the meeting and requests stage `j` into `free`, the stage's own place.
    // A row of MFMAs covers the reads of one x and one w fragment and, spread, a load or two: all of a step's loads at
    // once hold the wave at their issue while its matrix core idles (4096 x 4096 x 4096: 3 per row 59.8, 4 per row
    // 65.8 us, against 55.9).
    auto step = [&](bool second, const i32x4 (&x)[FM], const i32x4 (&w)[FN], const uint8_t* next, int at,
                    i32x4 (&xn)[FM], i32x4 (&wn)[FN], uint8_t* free, int j) __attribute__((always_inline)) {
        if (second) {
            wait_vm<(NS - 2) * NL>();                     // the next stage's loads have arrived ..
            __builtin_amdgcn_s_waitcnt(0xC07F);           // .. and lgkmcnt(0): this one's reads are done
            __builtin_amdgcn_s_barrier();
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < FN; ++n) {
            if (second) request(free, j, 0, n * NL / FN, (n + 1) * NL / FN);
            wn[n] = *(const i32x4*)(next + bw + at + n * 2048);
#pragma unroll
            for (int m = n * FM / FN; m < (n + 1) * FM / FN; ++m) xn[m] = *(const i32x4*)(next + bx + at + m * 2048);
#pragma unroll
            for (int m = 0; m < FM; ++m)
                acc[n][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[n], x[m], acc[n][m], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // both steps of the stage in `cur`, `next` the one after it; stage j + NS is requested
    auto stage = [&](uint8_t* cur, const uint8_t* next, int j) __attribute__((always_inline)) {
        step(false, fx0, fw0, cur, at1, fx1, fw1, nullptr, 0);
        step(true, fx1, fw1, next, at0, fx0, fw0, cur, j + NS);
    };
    auto mask = [&](i32x4 (&x)[FM], int left) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < FM; ++m) x[m] = 16 * q < left ? x[m] : i32x4{0, 0, 0, 0};
    };
    // a stage of the first turn: begins with the first stage's fragments, and masks its columns past Kin
    auto masked = [&](int place, int skip, uint8_t* cur, const uint8_t* next) __attribute__((always_inline)) {
        if (place < NS - 1 && place < skip) return;      // skip < NS
        const int j = place - skip, left = j == 0 ? valid : 128;
        if (j == 0) {
            wait_vm<(NS - 1) * NL>();
            __builtin_amdgcn_s_barrier();
#pragma unroll
            for (int n = 0; n < FN; ++n) fw0[n] = *(const i32x4*)(cur + bw + at0 + n * 2048);
#pragma unroll
            for (int m = 0; m < FM; ++m) fx0[m] = *(const i32x4*)(cur + bx + at0 + m * 2048);
        }
        mask(fx0, left);
        step(false, fx0, fw0, cur, at1, fx1, fw1, nullptr, 0);
        mask(fx1, left - 64);
        step(true, fx1, fw1, next, at0, fx0, fw0, cur, j + NS);
    };
    if (K > 0) {
        // turns of NS stages; the first may be short: it starts at place `skip` of the ring
        const int turns = (stages + NS - 1) / NS, skip = turns * NS - stages;
        // the first NS stages, in their order: loads return in it
        auto begin = [&](int place, uint8_t* st, bool wrapped) __attribute__((always_inline)) {
            if ((place < skip) != wrapped) return;
            // columns past Kin in the last block are read from its first chunk, a block past Kin is the one before it
            const bool first = !wrapped && place == skip, none = first && valid == 0;
            request(st, none ? 1 : place - skip + (wrapped ? NS : 0), first && !none && 16 * c >= valid ? 16 * c : 0, 0,
                    NL);
        };
        begin(0, st0, false);
        begin(1, st1, false);
        if constexpr (NS > 2) begin(2, st2, false);
        if constexpr (NS > 3) begin(3, st3, false);
        begin(0, st0, true);
        if constexpr (NS > 2) begin(1, st1, true);
        if constexpr (NS > 3) begin(2, st2, true);
        masked(0, skip, st0, st1);
        masked(1, skip, st1, NS > 2 ? st2 : st0);
        if constexpr (NS > 2) masked(2, skip, st2, NS > 3 ? st3 : st0);
        if constexpr (NS > 3) masked(3, skip, st3, st0);
        for (int j = NS - skip; j < stages; j += NS) {
            stage(st0, st1, j);
            stage(st1, NS > 2 ? st2 : st0, j + 1);
            if constexpr (NS > 2) stage(st2, NS > 3 ? st3 : st0, j + 2);
            if constexpr (NS > 3) stage(st3, st0, j + 3);
        }
        wait_vm<0>();     // the requests past the last stage: no load may land after the workgroup has left
    }
    if constexpr (KS > 1) {
        // the groups' sums meet in the stages' place (even tiles in the first's, odd ones in the second's): group g
        // adds up and stores the tiles g, g + KS, ..
        constexpr int HT = (FM * FN + 1) / 2;
        static_assert(4 * HT * 1024 <= STAGE, "partial sums fit the stages");
        __syncthreads();
        i32x4 *const red0 = (i32x4*)st0_, *const red1 = (i32x4*)st1_;
#pragma unroll
        for (int n = 0; n < FN; ++n)
#pragma unroll
            for (int m = 0; m < FM; ++m)
                ((n * FM + m) & 1 ? red1 : red0)[((group * 4 + wave) * HT + (n * FM + m) / 2) * 64 + lane] = acc[n][m];
        __syncthreads();
        const int mb = m0 + (wave & 1) * (16 * FM) + r, nb = n0 + (wave >> 1) * (16 * FN) + 4 * q;
        for (int t = group; t < FM * FN; t += KS) {
            const int mm = mb + 16 * (t % FM), nn = nb + 16 * (t / FM);
            if (mm >= A.M || nn >= A.N) continue;
            i32x4 sum = {0, 0, 0, 0};
#pragma unroll
            for (int g = 0; g < KS; ++g) sum += (t & 1 ? red1 : red0)[((g * 4 + wave) * HT + t / 2) * 64 + lane];
            const float xs = A.xs[mm];
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (float)sum[e] * (xs * A.ws[nn + e < A.N ? nn + e : A.N - 1]);
            store_quad<YT>(A.y, (int64_t)mm * A.N + nn, v, A.N - nn);
        }
        return;
    }
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

// ---------------------------------------------------------------------------
// The kernels, and which one a product takes: the one of the least estimate:
// `base` and a smooth maximum (the 8th root of the sum of 8th powers) of
//   rounds (setup + turn turns)     a workgroup's own latency,
//   q (wg + busy turns)             q workgroups' work on a compute unit,
//   stream bytes / 5.2e6            the operands and outputs, at memory's rate,
// with `turns` the 128-column blocks of one column group, `rounds` how often
// the resident workgroups are replaced and q the tiles of the fullest compute
// unit.  The constants are in microseconds, but fitted to the choice, not to
// each time: so that over the measured times of every kernel on 1397 products
// (M 1 .. 8192, N 150 .. 151936, Kin 128 .. 32768, half of them drawn at
// random; fp32 outputs, weights in no cache, as in a model that runs layer by
// layer) the choices cost least: 0.7% (geometric mean) against the fastest of
// these kernels, 17% at worst (43 x 801 x 2272).  A fit without half of the
// random products cost 1.2% on those.
struct Kernel {
    void (*f32)(Args, int, int);
    void (*bf16)(Args, int, int);
    int tm, tn;                  // tile
    int groups, threads;         // column groups of a workgroup
    int resident;                // workgroups on a compute unit
    double turn, setup, busy, wg, stream, base;
};
#define TQ_DENSE_FEW(W) {k_dense_i8_few<TQ_F32, W>, k_dense_i8_few<TQ_BF16, W>, 16, 16, W, 64 * W, 4
#define TQ_DENSE_TILE(FM, FN, KS, NS, RES)                                                                        \
    {k_dense_i8_tile<TQ_F32, FM, FN, KS, NS>, k_dense_i8_tile<TQ_BF16, FM, FN, KS, NS>, 32 * FM, 32 * FN, KS, \
     256 * KS, RES
const Kernel kKernels[] = {
    TQ_DENSE_FEW(4),              0.000, 0.000, 0.003, 0.000, 1.710, 1.540},     // M <= 16 only
    TQ_DENSE_TILE(1, 1, 1, 4, 5), 0.289, 0.896, 0.119, 1.050, 0.973, 0.209},
    TQ_DENSE_TILE(1, 1, 2, 4, 2), 0.378, 0.001, 0.318, 2.150, 0.000, 0.182},
    TQ_DENSE_TILE(1, 2, 2, 4, 1), 0.000, 6.510, 0.507, 0.557, 1.400, 0.436},
    TQ_DENSE_TILE(2, 2, 1, 3, 3), 0.374, 2.290, 0.380, 0.360, 0.521, 0.000},
    TQ_DENSE_TILE(2, 2, 2, 4, 1), 0.000, 6.800, 0.603, 2.660, 0.992, 0.417},
    TQ_DENSE_TILE(4, 2, 1, 3, 2), 0.012, 4.600, 0.402, 2.770, 1.000, 0.001},
    TQ_DENSE_TILE(4, 4, 1, 3, 1), 0.532, 0.852, 0.305, 4.240, 0.008, 0.715},
    TQ_DENSE_TILE(4, 8, 1, 3, 1), 0.680, 5.470, 0.659, 5.140, 0.013, 0.000},
    TQ_DENSE_TILE(6, 8, 1, 2, 1), 1.000, 3.770, 0.765, 7.280, 0.828, 0.000},
    TQ_DENSE_TILE(8, 8, 1, 2, 1), 0.954, 9.660, 1.200, 0.432, 0.034, 0.000},
};

int64_t tiles_of(const Kernel& k, int64_t M, int64_t N) { return ((M + k.tm - 1) / k.tm) * ((N + k.tn - 1) / k.tn); }

double estimate(const Kernel& k, int64_t M, int64_t N, int64_t Kin, int64_t y_bytes, int cus)
{
    const double x = (double)tiles_of(k, M, N) / cus;
    const double turns = (double)(((Kin + 127) / 128 + k.groups - 1) / k.groups);
    const double q = x <= k.resident || k.resident == 1 ? ceil(x) : x;
    const double own = ceil(x / k.resident) * (k.setup + k.turn * turns), work = q * (k.wg + k.busy * turns);
    const double mem = k.stream * (double)(N * Kin + M * Kin + y_bytes) / 5.2e6;
    const auto eighth = [](double v) { return v *= v, v *= v, v * v; };
    return k.base + sqrt(sqrt(sqrt(eighth(own) + eighth(work) + eighth(mem))));
}

// The kernel for a product, or null where no launch holds its tiles.
const Kernel* pick(int64_t M, int64_t N, int64_t Kin, int64_t y_bytes)
{
    const int cus = tq_device_cus();
    const Kernel* best = nullptr;
    double best_us = 0.0;
    for (size_t i = M <= 16 ? 0 : 1; i < sizeof kKernels / sizeof kKernels[0]; ++i) {
        const Kernel& k = kKernels[i];
        if (tiles_of(k, M, N) > (int64_t)UINT32_MAX / k.threads) continue;     // a launch counts its threads in 32 bits
        if (M <= 32 && k.tm >= 128) continue;     // mostly absent tokens: at most 10% faster anywhere, 8% slower on a
                                                  // head of 128256 rows where the estimates took one
        const double us = estimate(k, M, N, Kin, y_bytes, cus);
        if (!best || us < best_us) best = &k, best_us = us;
    }
    return best;
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
        return tq_fail(TQ_ERR_SHAPE,
                       "M = %lld, N = %lld, in_features = %lld: M and N up to %d, Kin a multiple of 16 up to %d",
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
    const Kernel* k = pick(M, N, Kin, yb);
    if (!k) return tq_fail(TQ_ERR_UNSUPPORTED, "%lld x %lld outputs exceed one launch", (long long)M, (long long)N);
    const Args A{xq, x_scale, w, w_scale, y, (int32_t)M, (int32_t)N, (int32_t)Kin};
    const int tm = (int)((M + k->tm - 1) / k->tm), tn = (int)((N + k->tn - 1) / k->tn);
    hipLaunchKernelGGL(y_type == TQ_F32 ? k->f32 : k->bf16, dim3((unsigned)((int64_t)tm * tn)), dim3(k->threads), 0,
                       (hipStream_t)stream, A, tm, tn);
    if ((s = tq_check_launch("tq_gemm_dense_i8"))) return s;
    return tq_ok();
}
