// libtq: tq_moe_dispatch, tq_moe_combine, tq_moe_combine_grad -- the rows of
// a mixture-of-experts layer, sorted by expert and brought back.
//
// The sort is a stable counting sort with n_experts + 1 buckets (the last
// one for pairs of no expert): how many pairs of each bucket stand before a
// wave's run of pairs, then each pair's rank inside its wave from ballots.
// No atomics on positions, so the order is the definition's.  The row copies
// and sums are bound by HBM: a token's row is read once and written to each
// of its places, or its top_k rows are read once and written as one.
#include "tq_internal.h"

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr int kSortThreads = 1024;            // one workgroup's sort
constexpr int64_t kSmallPairs = 8192;         // up to here one workgroup sorts ...
constexpr int kSmallExperts = 960;            // ... if its counters (16 waves by n_experts + 1) fit 64 KiB of LDS
constexpr int kBlockThreads = 256;            // the two-launch sort's workgroups
constexpr int64_t kBlockPairs = 2048;         // their pairs, at least
constexpr int kMaxBlocks = 256;
constexpr int kMaxGrid = 1 << 20;             // workgroups of one launch; more tokens are walked in a loop

// Lanes of the wave (active ones) whose bucket equals this lane's: one
// ballot per bit of the bucket.
__device__ __forceinline__ uint64_t match_bucket(int b, int bits, bool active)
{
    uint64_t m = __ballot(active);
    for (int i = 0; i < bits; ++i) {
        const uint64_t on = __ballot((b >> i) & 1);
        m &= ((b >> i) & 1) ? on : ~on;
    }
    return m;
}

__device__ __forceinline__ int bucket_of(const int32_t* experts, int64_t p, int E)
{
    const int e = experts[p];
    return e >= 0 && e < E ? e : E;
}

// Exclusive sum over the workgroup's threads; *total gets the whole sum.
template <int T>
__device__ __forceinline__ int block_scan(int v, int* total)
{
    __shared__ int wsum[T / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int s = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(s, off, 64);
        if (lane >= off) s += o;
    }
    if (lane == 63) wsum[wave] = s;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < T / 64; ++k) {
        const int w = wsum[k];
        before += k < wave ? w : 0;
        all += w;
    }
    *total = all;
    return before + s - v;
}

// The workgroup's pairs p0 .. p1 - 1, a contiguous run of them per wave;
// cnt[wave][bucket] (LDS) gets each run's counts.
template <int T>
__device__ __forceinline__ void run_of_wave(int64_t p0, int64_t p1, int64_t* a, int64_t* b)
{
    const int64_t len = (p1 - p0 + T / 64 * 64 - 1) / (T / 64 * 64) * 64;
    const int64_t at = p0 + (threadIdx.x >> 6) * len;
    *a = at < p1 ? at : p1;
    *b = at + len < p1 ? at + len : p1;
}

template <int T>
__device__ __forceinline__ void count_runs(const int32_t* experts, int64_t p0, int64_t p1, int E, int* cnt)
{
    for (int i = threadIdx.x; i < (T / 64) * (E + 1); i += T) cnt[i] = 0;
    __syncthreads();
    int64_t a, b;
    run_of_wave<T>(p0, p1, &a, &b);
    int* mine = cnt + (threadIdx.x >> 6) * (E + 1);
    for (int64_t p = a + (threadIdx.x & 63); p < b; p += 64) atomicAdd(&mine[bucket_of(experts, p, E)], 1);
    __syncthreads();
}

// cnt[wave][bucket] holds the first row of that run's pairs of the bucket;
// every pair takes the next one.
template <int T>
__device__ __forceinline__ void place_runs(const int32_t* experts, int64_t p0, int64_t p1, int E, int bits, int* cnt,
                                           int32_t* rows, int32_t* pairs)
{
    int64_t a, b;
    run_of_wave<T>(p0, p1, &a, &b);
    int* mine = cnt + (threadIdx.x >> 6) * (E + 1);
    const int lane = threadIdx.x & 63;
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    for (int64_t q = a; q < b; q += 64) {
        const int64_t p = q + lane;
        const bool on = p < b;
        const int e = on ? bucket_of(experts, p, E) : E;
        const uint64_t same = match_bucket(e, bits, on);
        if (on) {
            const int rank = __popcll(same & below);
            const int row = mine[e] + rank;
            rows[p] = e < E ? row : -1;
            pairs[row] = e < E ? (int32_t)p : -1;
        }
        // the bucket's first lane moves the counter on, after every lane has read it
        __builtin_amdgcn_wave_barrier();
        if (on && (same & below) == 0) mine[e] += __popcll(same);
        __builtin_amdgcn_wave_barrier();
    }
}

// One workgroup sorts every pair.
__global__ __launch_bounds__(kSortThreads) void k_sort_one(const int32_t* __restrict__ experts, int64_t P, int E, int bits,
                                                           int32_t* __restrict__ rows, int32_t* __restrict__ pairs,
                                                           int32_t* __restrict__ offsets)
{
    extern __shared__ int cnt[];
    constexpr int W = kSortThreads / 64;
    count_runs<kSortThreads>(experts, 0, P, E, cnt);
    const int e = threadIdx.x;                       // E <= kSortThreads buckets, one per thread
    int sum = 0;
    if (e < E)
        for (int w = 0; w < W; ++w) sum += cnt[w * (E + 1) + e];
    int total = 0;
    const int first = block_scan<kSortThreads>(sum, &total);
    if (e < E) {
        offsets[e] = first;
        int at = first;
        for (int w = 0; w < W; ++w) {
            const int c = cnt[w * (E + 1) + e];
            cnt[w * (E + 1) + e] = at;
            at += c;
        }
    }
    if (e == 0) {
        offsets[E] = total;
        int at = total;
        for (int w = 0; w < W; ++w) {
            const int c = cnt[w * (E + 1) + E];
            cnt[w * (E + 1) + E] = at;
            at += c;
        }
    }
    __syncthreads();
    place_runs<kSortThreads>(experts, 0, P, E, bits, cnt, rows, pairs);
}

// Two launches: each workgroup's counts, then the places.
__global__ __launch_bounds__(kBlockThreads) void k_sort_count(const int32_t* __restrict__ experts, int64_t P, int64_t per,
                                                              int E, int32_t* __restrict__ counts)
{
    extern __shared__ int cnt[];
    const int64_t p0 = blockIdx.x * per, p1 = p0 + per < P ? p0 + per : P;
    count_runs<kBlockThreads>(experts, p0, p1, E, cnt);
    for (int e = threadIdx.x; e <= E; e += kBlockThreads) {
        int s = 0;
        for (int w = 0; w < kBlockThreads / 64; ++w) s += cnt[w * (E + 1) + e];
        counts[blockIdx.x * (E + 1) + e] = s;
    }
}

__global__ __launch_bounds__(kBlockThreads) void k_sort_place(const int32_t* __restrict__ experts, int64_t P, int64_t per,
                                                              int E, int bits, const int32_t* __restrict__ counts,
                                                              int32_t* __restrict__ rows, int32_t* __restrict__ pairs,
                                                              int32_t* __restrict__ offsets)
{
    extern __shared__ int cnt[];
    constexpr int W = kBlockThreads / 64, PER = (kMaxExperts + kBlockThreads - 1) / kBlockThreads;
    const int64_t p0 = blockIdx.x * per, p1 = p0 + per < P ? p0 + per : P;
    count_runs<kBlockThreads>(experts, p0, p1, E, cnt);
    // thread i's buckets are i * n .. : their totals, and what stands before this workgroup
    const int n = (E + kBlockThreads - 1) / kBlockThreads;
    int before[PER], sum = 0, all[PER];
    for (int k = 0; k < PER; ++k) {
        const int e = threadIdx.x * n + k;
        before[k] = all[k] = 0;
        if (k < n && e < E)
            for (unsigned b = 0; b < gridDim.x; ++b) {
                const int c = counts[b * (E + 1) + e];
                all[k] += c;
                before[k] += b < blockIdx.x ? c : 0;
            }
        sum += all[k];
    }
    int total = 0;
    int first = block_scan<kBlockThreads>(sum, &total);
    for (int k = 0; k < PER; ++k) {
        const int e = threadIdx.x * n + k;
        if (k < n && e < E) {
            if (blockIdx.x == 0) offsets[e] = first;
            int at = first + before[k];
            for (int w = 0; w < W; ++w) {
                const int c = cnt[w * (E + 1) + e];
                cnt[w * (E + 1) + e] = at;
                at += c;
            }
        }
        first += all[k];
    }
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) offsets[E] = total;
        int at = total;
        for (unsigned b = 0; b < blockIdx.x; ++b) at += counts[b * (E + 1) + E];
        for (int w = 0; w < W; ++w) {
            const int c = cnt[w * (E + 1) + E];
            cnt[w * (E + 1) + E] = at;
            at += c;
        }
    }
    __syncthreads();
    place_runs<kBlockThreads>(experts, p0, p1, E, bits, cnt, rows, pairs);
}

// Copy each token's row to its places: T threads per token, 16 bytes per
// thread and step.
template <int T>
__global__ __launch_bounds__(256) void k_spread_rows(int64_t tokens, int top_k, int64_t row_units,
                                                     const int32_t* __restrict__ rows, const u32x4* __restrict__ x,
                                                     const float* __restrict__ x_scale, u32x4* __restrict__ xs,
                                                     float* __restrict__ xs_scale)
{
    constexpr int G = 256 / T;
    const int tid = threadIdx.x % T;
    for (int64_t t = (int64_t)blockIdx.x * G + threadIdx.x / T; t < tokens; t += (int64_t)gridDim.x * G) {
        const int32_t* r = rows + t * top_k;
        for (int64_t u = tid; u < row_units; u += T) {
            const u32x4 v = x[t * row_units + u];
            for (int j = 0; j < top_k; ++j)
                if (r[j] >= 0) xs[r[j] * row_units + u] = v;
        }
        if (x_scale)
            for (int j = tid; j < top_k; j += T)
                if (r[j] >= 0) xs_scale[r[j]] = x_scale[t];
    }
}

// U elements of a row as fp32, and back.
template <int TYPE, int U>
__device__ __forceinline__ void load_u(const void* base, int64_t unit, float* v)
{
    if (TYPE == TQ_F32) {
#pragma unroll
        for (int i = 0; i < U / 4; ++i) {
            const f32x4 f = ((const f32x4*)base)[unit * (U / 4) + i];
            v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
        }
    } else {
        uint32_t w[U / 2];
        if (U == 8) {
            const u32x4 q = ((const u32x4*)base)[unit];
            w[0] = q.x, w[1] = q.y, w[U / 2 - 2] = q.z, w[U / 2 - 1] = q.w;
        } else {
            const u32x2 q = ((const u32x2*)base)[unit];
            w[0] = q.x, w[1] = q.y;
        }
#pragma unroll
        for (int i = 0; i < U / 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const uint16_t lo = __builtin_bit_cast(uint16_t, (__bf16)a), hi = __builtin_bit_cast(uint16_t, (__bf16)b);
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

template <int TYPE, int U>
__device__ __forceinline__ void store_u(void* base, int64_t unit, const float* v)
{
    if (TYPE == TQ_F32) {
#pragma unroll
        for (int i = 0; i < U / 4; ++i)
            ((f32x4*)base)[unit * (U / 4) + i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    } else if (U == 8) {
        ((u32x4*)base)[unit] = u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[U - 4], v[U - 3]),
                                     bf16_pair(v[U - 2], v[U - 1])};
    } else {
        ((u32x2*)base)[unit] = u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    }
}

// A unit is 16 bytes of a ys row.
template <int TYPE>
constexpr int unit_of() { return TYPE == TQ_F32 ? 4 : 8; }

template <int ST, int YT, int T>
__global__ __launch_bounds__(256) void k_combine(int64_t tokens, int top_k, int64_t width, int64_t n_rows,
                                                 const int32_t* __restrict__ rows, const float* __restrict__ weights,
                                                 const void* __restrict__ ys, void* __restrict__ y)
{
    constexpr int U = unit_of<ST>(), G = 256 / T;
    const int tid = threadIdx.x % T;
    const int64_t units = width / U;
    for (int64_t t = (int64_t)blockIdx.x * G + threadIdx.x / T; t < tokens; t += (int64_t)gridDim.x * G) {
        for (int64_t u = tid; u < units; u += T) {
            float acc[U] = {};
            for (int j = 0; j < top_k; ++j) {
                const int64_t r = rows[t * top_k + j];
                if (r < 0 || r >= n_rows) continue;
                const float w = weights ? weights[t * top_k + j] : 1.0f;
                float v[U];
                load_u<ST, U>(ys, r * units + u, v);
#pragma unroll
                for (int i = 0; i < U; ++i) acc[i] = fmaf(w, v[i], acc[i]);
            }
            store_u<YT, U>(y, t * units + u, acc);
        }
    }
}

// One workgroup per token: d_ys rows and the dot products, pair by pair.
template <int DT, int ST>
__global__ __launch_bounds__(256) void k_combine_grad(int64_t tokens, int top_k, int64_t width, int64_t n_rows,
                                                      const int32_t* __restrict__ rows,
                                                      const float* __restrict__ weights, const void* __restrict__ dy,
                                                      const void* __restrict__ ys, void* __restrict__ d_ys,
                                                      float* __restrict__ d_weights)
{
    constexpr int U = unit_of<ST>();
    __shared__ float red[4];
    const int64_t units = width / U;
    for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
        for (int j = 0; j < top_k; ++j) {
            const int64_t r = rows[t * top_k + j];
            const bool on = r >= 0 && r < n_rows;
            float dot = 0.0f;
            if (on) {
                const float w = weights ? weights[t * top_k + j] : 1.0f;
                for (int64_t u = threadIdx.x; u < units; u += 256) {
                    float g[U], v[U];
                    load_u<DT, U>(dy, t * units + u, g);
                    if (d_weights) {
                        load_u<ST, U>(ys, r * units + u, v);
#pragma unroll
                        for (int i = 0; i < U; ++i) dot = fmaf(g[i], v[i], dot);
                    }
                    if (d_ys) {
#pragma unroll
                        for (int i = 0; i < U; ++i) g[i] *= w;
                        store_u<ST, U>(d_ys, r * units + u, g);
                    }
                }
            }
            if (d_weights) {
#pragma unroll
                for (int off = 32; off > 0; off >>= 1) dot += __shfl_xor(dot, off, 64);
                if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = dot;
                __syncthreads();
                if (threadIdx.x == 0) d_weights[t * top_k + j] = (red[0] + red[1]) + (red[2] + red[3]);
                __syncthreads();
            }
        }
    }
}

int64_t size_of(int t) { return t == TQ_F32 ? 4 : t == TQ_BF16 ? 2 : 1; }

// Sizes shared by the three calls.
tq_status check_sizes(int64_t tokens, int32_t top_k, int64_t width)
{
    if (tokens < 0 || width < 0) return tq_fail(TQ_ERR_ARG, "negative size tokens = %lld, width = %lld",
                                                (long long)tokens, (long long)width);
    if (top_k < 1 || top_k > kMaxTopK) return tq_fail(TQ_ERR_ARG, "top_k = %d, must be 1..%d", top_k, kMaxTopK);
    if (width % 16 || width > TQ_MAX_KIN)
        return tq_fail(TQ_ERR_SHAPE, "width = %lld, must be a multiple of 16 up to %d", (long long)width, TQ_MAX_KIN);
    if (tokens > ((int64_t)1 << 30) / top_k)
        return tq_fail(TQ_ERR_SHAPE, "tokens * top_k = %lld * %d exceeds 2^30", (long long)tokens, top_k);
    return TQ_OK;
}

tq_status check_float_type(int32_t t, const char* name)
{
    if (t != TQ_F32 && t != TQ_BF16) return tq_fail(TQ_ERR_ARG, "%s = %d, must be TQ_F32 or TQ_BF16", name, t);
    return TQ_OK;
}

// One array of a call, for the overlap checks.
struct Span {
    const void* p;
    int64_t bytes;
    const char* name;
};

// Every output against every input and every other output.
template <int NO, int NI>
tq_status check_spans(const Span (&out)[NO], const Span (&in)[NI])
{
    tq_status s;
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if ((s = tq_check_overlap(out[i].p, out[i].bytes, out[i].name, in[j].p, in[j].bytes, in[j].name))) return s;
        for (int j = 0; j < i; ++j)
            if ((s = tq_check_overlap(out[i].p, out[i].bytes, out[i].name, out[j].p, out[j].bytes, out[j].name)))
                return s;
    }
    return TQ_OK;
}

unsigned grid_of(int64_t tokens, int per)
{
    const int64_t n = (tokens + per - 1) / per;
    return (unsigned)(n < kMaxGrid ? n : kMaxGrid);
}

// Workgroups and pairs per workgroup of the two-launch sort.
int64_t sort_blocks(int64_t P, int64_t* per)
{
    int64_t n = (P + kBlockPairs - 1) / kBlockPairs;
    if (n > kMaxBlocks) n = kMaxBlocks;
    *per = n ? (P + n - 1) / n : 0;
    return n;
}

}  // namespace

TQ_EXPORT tq_status tq_moe_dispatch_workspace_size(int64_t tokens, int32_t top_k, int32_t n_experts, size_t* bytes)
{
    tq_status s = check_sizes(tokens, top_k, 0);
    if (s) return s;
    if (!bytes) return tq_fail(TQ_ERR_ARG, "bytes is NULL");
    if (n_experts < 1 || n_experts > kMaxExperts)
        return tq_fail(TQ_ERR_ARG, "n_experts = %d, must be 1..%d", n_experts, kMaxExperts);
    const int64_t P = tokens * top_k;
    int64_t per;
    *bytes = P <= kSmallPairs && n_experts <= kSmallExperts ? 0 : (size_t)tq_align256(sort_blocks(P, &per) * (n_experts + 1) * 4);
    return tq_ok();
}

TQ_EXPORT tq_status tq_moe_dispatch(int64_t tokens, int32_t top_k, int32_t n_experts, const int32_t* experts,
                                    int32_t* rows, int32_t* pairs, int32_t* offsets, int64_t width, int32_t x_type,
                                    const void* x, const float* x_scale, void* xs, float* xs_scale, void* workspace,
                                    size_t workspace_bytes, void* stream)
{
    tq_status s;
    size_t need = 0;
    if ((s = tq_moe_dispatch_workspace_size(tokens, top_k, n_experts, &need))) return s;
    if ((s = check_sizes(tokens, top_k, width))) return s;
    if (x && x_type != TQ_F32 && x_type != TQ_BF16 && x_type != TQ_I8)
        return tq_fail(TQ_ERR_ARG, "x_type = %d, must be TQ_F32, TQ_BF16 or TQ_I8", x_type);
    const int64_t P = tokens * top_k;
    if ((s = tq_check_ptr(offsets, "offsets", false, 4))) return s;
    if ((s = tq_check_ptr(experts, "experts", P == 0, 4))) return s;
    if ((s = tq_check_ptr(rows, "rows", P == 0, 4))) return s;
    if ((s = tq_check_ptr(pairs, "pairs", P == 0, 4))) return s;
    const bool copy = x && P > 0 && width > 0, scales = x && x_type == TQ_I8;
    if (copy) {
        if ((s = tq_check_ptr(x, "x", false))) return s;
        if ((s = tq_check_ptr(xs, "xs", false))) return s;
    }
    if (scales && P > 0) {
        if ((s = tq_check_ptr(x_scale, "x_scale", false, 4))) return s;
        if ((s = tq_check_ptr(xs_scale, "xs_scale", false, 4))) return s;
    }
    if ((s = tq_check_ptr(workspace, "workspace", need == 0))) return s;
    if (workspace_bytes < need)
        return tq_fail(TQ_ERR_ARG, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    const int64_t row_bytes = copy ? width * size_of(x_type) : 0;
    const Span out[] = {{rows, P * 4, "rows"}, {pairs, P * 4, "pairs"}, {offsets, (n_experts + 1) * 4, "offsets"},
                        {xs, P * row_bytes, "xs"}, {xs_scale, scales ? P * 4 : 0, "xs_scale"},
                        {workspace, (int64_t)need, "workspace"}};
    const Span in[] = {{experts, P * 4, "experts"}, {x, tokens * row_bytes, "x"},
                       {x_scale, scales ? tokens * 4 : 0, "x_scale"}};
    if ((s = check_spans(out, in))) return s;
    hipStream_t st = (hipStream_t)stream;
    int bits = 1;
    while ((1 << bits) <= n_experts) ++bits;
    if (need == 0) {
        hipLaunchKernelGGL(k_sort_one, dim3(1), dim3(kSortThreads), kSortThreads / 64 * (n_experts + 1) * 4, st, experts,
                           P, n_experts, bits, rows, pairs, offsets);
    } else {
        int64_t per;
        const unsigned n = (unsigned)sort_blocks(P, &per);
        const size_t lds = kBlockThreads / 64 * (n_experts + 1) * 4;
        hipLaunchKernelGGL(k_sort_count, dim3(n), dim3(kBlockThreads), lds, st, experts, P, per, n_experts,
                           (int32_t*)workspace);
        hipLaunchKernelGGL(k_sort_place, dim3(n), dim3(kBlockThreads), lds, st, experts, P, per, n_experts, bits,
                           (const int32_t*)workspace, rows, pairs, offsets);
    }
    if ((s = tq_check_launch("tq_moe_dispatch sort"))) return s;
    if (copy || (scales && P > 0)) {
        const int64_t units = width * size_of(x_type) / 16;
        const float* xsc = scales ? x_scale : nullptr;
        if (units <= 256)
            hipLaunchKernelGGL(k_spread_rows<64>, dim3(grid_of(tokens, 4)), dim3(256), 0, st, tokens, top_k, units, rows,
                               (const u32x4*)x, xsc, (u32x4*)xs, xs_scale);
        else
            hipLaunchKernelGGL(k_spread_rows<256>, dim3(grid_of(tokens, 1)), dim3(256), 0, st, tokens, top_k, units,
                               rows, (const u32x4*)x, xsc, (u32x4*)xs, xs_scale);
        if ((s = tq_check_launch("tq_moe_dispatch rows"))) return s;
    }
    return tq_ok();
}

namespace {

template <int ST, int YT>
void launch_combine(int64_t tokens, int top_k, int64_t width, int64_t n_rows, const int32_t* rows, const float* weights,
                    const void* ys, void* y, hipStream_t st)
{
    if (width / unit_of<ST>() <= 256)
        hipLaunchKernelGGL((k_combine<ST, YT, 64>), dim3(grid_of(tokens, 4)), dim3(256), 0, st, tokens, top_k, width,
                           n_rows, rows, weights, ys, y);
    else
        hipLaunchKernelGGL((k_combine<ST, YT, 256>), dim3(grid_of(tokens, 1)), dim3(256), 0, st, tokens, top_k, width,
                           n_rows, rows, weights, ys, y);
}

template <int DT, int ST>
void launch_grad(int64_t tokens, int top_k, int64_t width, int64_t n_rows, const int32_t* rows, const float* weights,
                 const void* dy, const void* ys, void* d_ys, float* d_weights, hipStream_t st)
{
    hipLaunchKernelGGL((k_combine_grad<DT, ST>), dim3(grid_of(tokens, 1)), dim3(256), 0, st, tokens, top_k, width, n_rows,
                       rows, weights, dy, ys, d_ys, d_weights);
}

}  // namespace

TQ_EXPORT tq_status tq_moe_combine(int64_t tokens, int32_t top_k, int64_t width, int64_t n_rows, const int32_t* rows,
                                   const float* weights, int32_t ys_type, const void* ys, int32_t y_type, void* y,
                                   void* stream)
{
    tq_status s;
    if ((s = check_sizes(tokens, top_k, width))) return s;
    if ((s = check_float_type(ys_type, "ys_type")) || (s = check_float_type(y_type, "y_type"))) return s;
    if (n_rows < 0 || n_rows > INT32_MAX) return tq_fail(TQ_ERR_ARG, "n_rows = %lld", (long long)n_rows);
    if (tokens == 0 || width == 0) return tq_ok();
    if ((s = tq_check_ptr(rows, "rows", false, 4))) return s;
    if ((s = tq_check_ptr(weights, "weights", true, 4))) return s;
    if ((s = tq_check_ptr(ys, "ys", n_rows == 0))) return s;
    if ((s = tq_check_ptr(y, "y", false))) return s;
    const int64_t P = tokens * top_k;
    const Span out[] = {{y, tokens * width * size_of(y_type), "y"}};
    const Span in[] = {{rows, P * 4, "rows"}, {weights, P * 4, "weights"}, {ys, n_rows * width * size_of(ys_type), "ys"}};
    if ((s = check_spans(out, in))) return s;
    auto* fn = ys_type == TQ_F32 ? (y_type == TQ_F32 ? launch_combine<TQ_F32, TQ_F32> : launch_combine<TQ_F32, TQ_BF16>)
                                 : (y_type == TQ_F32 ? launch_combine<TQ_BF16, TQ_F32> : launch_combine<TQ_BF16, TQ_BF16>);
    fn(tokens, top_k, width, n_rows, rows, weights, ys, y, (hipStream_t)stream);
    if ((s = tq_check_launch("tq_moe_combine"))) return s;
    return tq_ok();
}

TQ_EXPORT tq_status tq_moe_combine_grad(int64_t tokens, int32_t top_k, int64_t width, int64_t n_rows,
                                        const int32_t* rows, const float* weights, int32_t dy_type, const void* dy,
                                        int32_t ys_type, const void* ys, void* d_ys, float* d_weights, void* stream)
{
    tq_status s;
    if ((s = check_sizes(tokens, top_k, width))) return s;
    if ((s = check_float_type(dy_type, "dy_type")) || (s = check_float_type(ys_type, "ys_type"))) return s;
    if (n_rows < 0 || n_rows > INT32_MAX) return tq_fail(TQ_ERR_ARG, "n_rows = %lld", (long long)n_rows);
    if (tokens == 0 || (!d_ys && !d_weights)) return tq_ok();
    if ((s = tq_check_ptr(rows, "rows", false, 4))) return s;
    if ((s = tq_check_ptr(weights, "weights", true, 4))) return s;
    if ((s = tq_check_ptr(dy, "dy", width == 0))) return s;
    if ((s = tq_check_ptr(ys, "ys", !d_weights || n_rows == 0 || width == 0))) return s;
    if ((s = tq_check_ptr(d_ys, "d_ys", true))) return s;
    if ((s = tq_check_ptr(d_weights, "d_weights", true, 4))) return s;
    const int64_t P = tokens * top_k, row = width * size_of(ys_type);
    const Span out[] = {{d_ys, n_rows * row, "d_ys"}, {d_weights, P * 4, "d_weights"}};
    const Span in[] = {{rows, P * 4, "rows"}, {weights, P * 4, "weights"}, {dy, tokens * width * size_of(dy_type), "dy"},
                       {ys, d_weights ? n_rows * row : 0, "ys"}};
    if ((s = check_spans(out, in))) return s;
    auto* fn = dy_type == TQ_F32 ? (ys_type == TQ_F32 ? launch_grad<TQ_F32, TQ_F32> : launch_grad<TQ_F32, TQ_BF16>)
                                 : (ys_type == TQ_F32 ? launch_grad<TQ_BF16, TQ_F32> : launch_grad<TQ_BF16, TQ_BF16>);
    fn(tokens, top_k, width, n_rows, rows, weights, dy, ys, d_ys, d_weights, (hipStream_t)stream);
    if ((s = tq_check_launch("tq_moe_combine_grad"))) return s;
    return tq_ok();
}
