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
constexpr int64_t kSmallPairs = 5120;         // up to here one workgroup sorts (4096 pairs 10.0 us with their rows of
                                              // 1 KiB, in two launches 11.1; 5600 pairs 11.2 against 10.5) ...
constexpr int kSmallExperts = 960;            // ... if its counters (16 waves by n_experts + 1) fit 64 KiB of LDS
constexpr int64_t kBlockPairs = 2048;         // the two-launch sort's pairs per workgroup, at least: with 1024 threads
constexpr int kMaxBlocks = 256;               // 65536 pairs take 10 us (256 threads and 1024 pairs: 13 us)
constexpr int kChunk = 2;                     // loads of ids at once in the sorts (4 measured alike, 8 slower)
constexpr int kMaxGrid = 1 << 20;             // workgroups of one launch; more tokens are walked in a loop
constexpr int64_t kFewPairs = 1024;           // up to here every wave finds its own rows (128 tokens, top 8: 5.4 us,
                                              // 9.3 us with a sort first; 256 tokens 8.3 against 8.9 us, but the
                                              // longer key list costs the smaller batches 1 us)

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

__device__ __forceinline__ int bucket(int e, int E) { return e >= 0 && e < E ? e : E; }
__device__ __forceinline__ int bucket_of(const int32_t* experts, int64_t p, int E) { return bucket(experts[p], E); }

// The lane's ids of the 64 kChunk pairs from q on, loaded at once (from b on
// the last one's before b).
__device__ __forceinline__ void load_chunk(const int32_t* experts, int64_t q, int64_t b, int (&e)[kChunk])
{
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        const int64_t p = q + 64 * i + (threadIdx.x & 63);
        e[i] = experts[p < b ? p : b - 1];
    }
}

// A bucket's counts per wave become the first rows of each wave's pairs, from
// `at` on (all read before any is written: one latency).
template <int W>
__device__ __forceinline__ void firsts_of(int* cnt, int E, int e, int at)
{
    int c[W];
#pragma unroll
    for (int w = 0; w < W; ++w) c[w] = cnt[w * (E + 1) + e];
#pragma unroll
    for (int w = 0; w < W; ++w) {
        cnt[w * (E + 1) + e] = at;
        at += c[w];
    }
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
    const int lane = threadIdx.x & 63;
    for (int64_t q = a; q < b; q += 64 * kChunk) {
        int e[kChunk];
        load_chunk(experts, q, b, e);
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            if (q + 64 * i + lane < b) atomicAdd(&mine[bucket(e[i], E)], 1);
    }
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
    for (int64_t c = a; c < b; c += 64 * kChunk) {
        int ids[kChunk];
        load_chunk(experts, c, b, ids);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            const int64_t q = c + 64 * i, p = q + lane;
            if (q >= b) break;
            const bool on = p < b;
            const int e = bucket(ids[i], E);
            const uint64_t same = match_bucket(e, bits, on);
            if (on) {
                const int rank = __popcll(same & below);
                const int row = mine[e] + rank;
                rows[p] = e < E ? row : -1;
                pairs[row] = e < E ? (int32_t)p : -1;
            }
            // the bucket's first lane moves the counter on, after every lane has read it and before any reads it again
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (on && (same & below) == 0) mine[e] += __popcll(same);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    }
}

// One workgroup sorts every pair.
__global__ __launch_bounds__(kSortThreads) void k_sort_one(const int32_t* __restrict__ experts, int64_t P, int E,
                                                           int bits, int32_t* __restrict__ rows,
                                                           int32_t* __restrict__ pairs, int32_t* __restrict__ offsets)
{
    extern __shared__ int cnt[];
    constexpr int W = kSortThreads / 64;
    count_runs<kSortThreads>(experts, 0, P, E, cnt);
    const int e = threadIdx.x;                       // E <= kSortThreads buckets, one per thread
    int sum = 0;
    if (e < E)
#pragma unroll
        for (int w = 0; w < W; ++w) sum += cnt[w * (E + 1) + e];
    int total = 0;
    const int first = block_scan<kSortThreads>(sum, &total);
    if (e < E) {
        offsets[e] = first;
        firsts_of<W>(cnt, E, e, first);
    }
    static_assert(kSmallExperts < kSortThreads, "the last thread has no expert");
    if (e == kSortThreads - 1) {
        offsets[E] = total;
        firsts_of<W>(cnt, E, E, total);
    }
    __syncthreads();
    place_runs<kSortThreads>(experts, 0, P, E, bits, cnt, rows, pairs);
}

// Two launches: each workgroup's counts (counts[bucket][workgroup], so that a
// bucket's are read 16 bytes at a time), then the places.
template <int T>
__global__ __launch_bounds__(T) void k_sort_count(const int32_t* __restrict__ experts, int64_t P, int64_t per, int E,
                                                  int32_t* __restrict__ counts)
{
    extern __shared__ int cnt[];
    const int64_t p0 = blockIdx.x * per < P ? blockIdx.x * per : P, p1 = p0 + per < P ? p0 + per : P;
    count_runs<T>(experts, p0, p1, E, cnt);
    for (int e = threadIdx.x; e <= E; e += T) {
        int s = 0;
#pragma unroll
        for (int w = 0; w < T / 64; ++w) s += cnt[w * (E + 1) + e];
        counts[(int64_t)e * gridDim.x + blockIdx.x] = s;
    }
}

template <int T>
__global__ __launch_bounds__(T) void k_sort_place(const int32_t* __restrict__ experts, int64_t P, int64_t per, int E,
                                                  int bits, const int32_t* __restrict__ counts,
                                                  int32_t* __restrict__ rows, int32_t* __restrict__ pairs,
                                                  int32_t* __restrict__ offsets)
{
    extern __shared__ int cnt[];
    constexpr int W = T / 64, PER = kMaxExperts / T;
    const int64_t p0 = blockIdx.x * per < P ? blockIdx.x * per : P, p1 = p0 + per < P ? p0 + per : P;
    count_runs<T>(experts, p0, p1, E, cnt);
    // thread i's buckets are i * n .. : their totals, and what stands before this workgroup
    const int n = (E + T - 1) / T, me = blockIdx.x;
    const int4* counts4 = (const int4*)counts;
    auto sums = [&](int e, int* all, int* before) {
        int a = 0, f = 0;
#pragma unroll 8
        for (int b = 0; b < (int)gridDim.x; b += 4) {
            const int4 c = counts4[((int64_t)e * gridDim.x + b) >> 2];
            a += c.x + c.y + c.z + c.w;
            f += (b < me ? c.x : 0) + (b + 1 < me ? c.y : 0) + (b + 2 < me ? c.z : 0) + (b + 3 < me ? c.w : 0);
        }
        *all = a, *before = f;
    };
    int before[PER], sum = 0, all[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int e = threadIdx.x * n + k;
        before[k] = all[k] = 0;
        if (k < n && e < E) sums(e, &all[k], &before[k]);
        sum += all[k];
    }
    int total = 0;
    int first = block_scan<T>(sum, &total);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int e = threadIdx.x * n + k;
        if (k < n && e < E) {
            if (me == 0) offsets[e] = first;
            firsts_of<W>(cnt, E, e, first + before[k]);
        }
        first += all[k];
    }
    if (threadIdx.x == T - 1) {
        if (me == 0) offsets[E] = total;
        int none, at;
        sums(E, &none, &at);
        firsts_of<W>(cnt, E, E, total + at);
    }
    __syncthreads();
    place_runs<T>(experts, p0, p1, E, bits, cnt, rows, pairs);
}

// In the row kernels a wave has one token and a run of 64 (k_combine: 64 V)
// units of 16 bytes of its row; a workgroup's 4 waves have 4 / W tokens and W
// neighbouring runs (W = 1 << lw; a row's runs at the same time, or memory
// pages are opened for each), blockIdx.y the next W.  The token is the same
// in all lanes, and told so to the compiler: row numbers and weights come
// through scalar loads.
__device__ __forceinline__ int64_t first_token(int lw)
{
    return ((int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) >> lw;
}
__device__ __forceinline__ int64_t token_step(int lw) { return (int64_t)gridDim.x * 4 >> lw; }
__device__ __forceinline__ int run_of(int lw)
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    return ((int)blockIdx.y << lw) + (wave & ((1 << lw) - 1));
}

// Copy each token's row to its places: read once, written top_k times, one
// unit per lane (2 and 4 were slower).  8192 tokens (5% of them padding), top
// 8, 2048 bf16: 51 us, 5.6 TB/s, and 61 us with the sort.
__global__ __launch_bounds__(256) void k_spread_rows(int64_t tokens, int top_k, int64_t units, int lw,
                                                     const int32_t* __restrict__ rows, const u32x4* __restrict__ x,
                                                     const float* __restrict__ x_scale, u32x4* __restrict__ xs,
                                                     float* __restrict__ xs_scale)
{
    const int lane = threadIdx.x & 63;
    const int run = run_of(lw);
    const int64_t u = run * 64 + lane;
    for (int64_t t = first_token(lw); t < tokens; t += token_step(lw)) {
        const int32_t* r = rows + t * top_k;
        if (u < units) {
            const u32x4 v = x[t * units + u];
            for (int j = 0; j < top_k; ++j)
                if (r[j] >= 0) __builtin_nontemporal_store(v, &xs[r[j] * units + u]);
        }
        if (x_scale && run == 0 && lane < top_k && r[lane] >= 0) xs_scale[r[lane]] = x_scale[t];
    }
}

// Sort and copy in one launch, for few pairs (64 B at most).  A pair's row is
// how many pairs have a smaller key bucket * P + pair: every wave counts that
// for its own token's pairs, 64 keys per ballot, with all keys loaded at once
// (64 tokens, top 8: 4.4 us, 5.8 us with four loads at a time; with B = 16 in
// place of 8 4.8 us).  The last workgroup finds the offsets.
template <int B>
__global__ __launch_bounds__(256) void k_dispatch_few(const int32_t* __restrict__ experts, int tokens, int top_k, int E,
                                                      int32_t* __restrict__ rows, int32_t* __restrict__ pairs,
                                                      int32_t* __restrict__ offsets, int64_t units, int lw,
                                                      const u32x4* __restrict__ x, const float* __restrict__ x_scale,
                                                      u32x4* __restrict__ xs, float* __restrict__ xs_scale)
{
    const int P = tokens * top_k, lane = threadIdx.x & 63;
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y != 0) return;
        __shared__ int cnt[kMaxExperts];
        constexpr int PER = kMaxExperts / 256;
        for (int e = threadIdx.x; e < kMaxExperts; e += 256) cnt[e] = 0;
        __syncthreads();
        for (int p = threadIdx.x; p < P; p += 256) {
            const int e = bucket_of(experts, p, E);
            if (e < E) atomicAdd(&cnt[e], 1);
        }
        __syncthreads();
        int own[PER], sum = 0, total = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) sum += own[k] = cnt[threadIdx.x * PER + k];
        int first = block_scan<256>(sum, &total);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if ((int)threadIdx.x * PER + k < E) offsets[threadIdx.x * PER + k] = first;
            first += own[k];
        }
        if (threadIdx.x == 0) offsets[E] = total;
        return;
    }
    const int t = (int)first_token(lw), run = run_of(lw);
    if (t >= tokens) return;
    const int64_t u = run * 64 + lane;
    u32x4 v = {0, 0, 0, 0};
    if (u < units) v = x[t * units + u];
    constexpr int J = 8;
    int k[B];
#pragma unroll
    for (int b = 0; b < B; ++b) k[b] = experts[b * 64 + lane < P ? b * 64 + lane : P - 1];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const int p = b * 64 + lane;
        k[b] = p < P ? bucket(k[b], E) * P + p : INT32_MAX;
    }
    for (int j0 = 0; j0 < top_k; j0 += J) {
        int key[J], row[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int p = t * top_k + (j0 + j < top_k ? j0 + j : 0);
            key[j] = bucket_of(experts, p, E) * P + p;
            row[j] = 0;
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (b * 64 < P)
#pragma unroll
                for (int j = 0; j < J; ++j) row[j] += __popcll(__ballot(k[b] < key[j]));
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (j0 + j >= top_k) break;
            const int p = t * top_k + j0 + j;
            const bool used = key[j] < E * P;
            if (run == 0 && lane == 0) {
                rows[p] = used ? row[j] : -1;
                pairs[row[j]] = used ? p : -1;
                if (x_scale && used) xs_scale[row[j]] = x_scale[t];
            }
            if (used && u < units) __builtin_nontemporal_store(v, &xs[row[j] * units + u]);
        }
    }
}

// 16 bytes of a row as fp32 values.
template <int TYPE, int U>
__device__ __forceinline__ void unpack(u32x4 q, float (&v)[U])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == TQ_F32) {
            v[i] = __uint_as_float(q[i]);
        } else {
            v[2 * i] = __uint_as_float(q[i] << 16);
            v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
        }
    }
}

// U elements of a row as fp32, and back (outputs are not read again here:
// stored non-temporally).
template <int TYPE, int U>
__device__ __forceinline__ void load_u(const void* base, int64_t unit, float (&v)[U])
{
    if constexpr (TYPE == TQ_F32) {
#pragma unroll
        for (int i = 0; i < U / 4; ++i) {
            const f32x4 f = ((const f32x4*)base)[unit * (U / 4) + i];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * i + e] = f[e];
        }
    } else if constexpr (U == 8) {
        unpack<TYPE, U>(((const u32x4*)base)[unit], v);
    } else {
        const u32x2 q = ((const u32x2*)base)[unit];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[2 * i] = __uint_as_float(q[i] << 16);
            v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const uint16_t lo = __builtin_bit_cast(uint16_t, (__bf16)a), hi = __builtin_bit_cast(uint16_t, (__bf16)b);
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

template <int TYPE, int U>
__device__ __forceinline__ void store_u(void* base, int64_t unit, const float (&v)[U])
{
    if constexpr (TYPE == TQ_F32) {
#pragma unroll
        for (int i = 0; i < U / 4; ++i)
            __builtin_nontemporal_store(f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]},
                                        &((f32x4*)base)[unit * (U / 4) + i]);
    } else if constexpr (U == 8) {
        __builtin_nontemporal_store(u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                                          bf16_pair(v[6], v[7])},
                                    &((u32x4*)base)[unit]);
    } else {
        __builtin_nontemporal_store(u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}, &((u32x2*)base)[unit]);
    }
}

// A unit is 16 bytes of a ys row.
template <int TYPE>
constexpr int unit_of() { return TYPE == TQ_F32 ? 4 : 8; }

// The rows of J pairs of one token (uniform): bit j of `ok` if pair j has one;
// the others' loads go to one that has (`ok` 0: nothing may be loaded).
template <int J>
struct Rows {
    int r[J];
    uint32_t ok;
};

template <int J>
__device__ __forceinline__ Rows<J> rows_of(const int32_t* rows, int j0, int top_k, int64_t n_rows)
{
    Rows<J> R;
    R.ok = 0;
    int some = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        R.r[j] = j0 + j < top_k ? rows[j0 + j] : -1;
        if (R.r[j] >= 0 && R.r[j] < n_rows) some = R.r[j], R.ok |= 1u << j;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
        if (!(R.ok >> j & 1)) R.r[j] = some;
    return R;
}

// y[t] = sum of weights times rows: J rows of 64 V units in flight per wave,
// each read once, so memory bounds it.
template <int ST, int YT, int J, int V>
__global__ __launch_bounds__(256) void k_combine(int64_t tokens, int top_k, int64_t units, int lw, int64_t n_rows,
                                                 const int32_t* __restrict__ rows, const float* __restrict__ weights,
                                                 const void* __restrict__ ys, void* __restrict__ y)
{
    constexpr int U = unit_of<ST>();
    const int lane = threadIdx.x & 63;
    const int64_t u = run_of(lw) * 64 * V + lane;
    for (int64_t t = first_token(lw); t < tokens; t += token_step(lw)) {
        float acc[V][U] = {};
        for (int j0 = 0; j0 < top_k; j0 += J) {
            const Rows<J> R = rows_of<J>(rows + t * top_k, j0, top_k, n_rows);
            if (!R.ok) continue;
            u32x4 v[J][V];
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (u + 64 * k < units) v[j][k] = ((const u32x4*)ys)[(int64_t)R.r[j] * units + u + 64 * k];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!(R.ok >> j & 1)) continue;
                const float w = weights ? weights[t * top_k + j0 + j] : 1.0f;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float f[U];
                    unpack<ST, U>(v[j][k], f);
#pragma unroll
                    for (int i = 0; i < U; ++i) acc[k][i] = fmaf(w, f[i], acc[k][i]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (u + 64 * k < units) store_u<YT, U>(y, t * units + u + 64 * k, acc[k]);
    }
}

// Sum each of 8 values over the wave: halves of the values change places with
// halves of the lanes, so 10 exchanges in place of 48.  Lane l gets the sum of
// value l / 8.
__device__ __forceinline__ float wave_sum8(const float (&v)[8])
{
    const int lane = threadIdx.x & 63;
    float a[4], b[2], c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool hi = lane & 32;
        a[i] = (hi ? v[i + 4] : v[i]) + __shfl_xor(hi ? v[i] : v[i + 4], 32, 64);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool hi = lane & 16;
        b[i] = (hi ? a[i + 2] : a[i]) + __shfl_xor(hi ? a[i] : a[i + 2], 16, 64);
    }
    const bool hi = lane & 8;
    c = (hi ? b[1] : b[0]) + __shfl_xor(hi ? b[0] : b[1], 8, 64);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) c += __shfl_xor(c, off, 64);
    return c;
}

// The gradient of k_combine: W waves per token walk its row 64 units each at
// a time; every unit of dy meets those of 8 rows, whose gradients are stored
// and whose dot products gather per lane until the row's end.
template <int DT, int ST, int W>
__global__ __launch_bounds__(256) void k_combine_grad(int64_t tokens, int top_k, int64_t units, int64_t n_rows,
                                                      const int32_t* __restrict__ rows,
                                                      const float* __restrict__ weights, const void* __restrict__ dy,
                                                      const void* __restrict__ ys, void* __restrict__ d_ys,
                                                      float* __restrict__ d_weights)
{
    constexpr int U = unit_of<ST>(), J = 8, G = 4 / W;
    __shared__ float red[4][J];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = wave % W;
    // with W > 1 (barriers) G is 1: all waves of the workgroup walk the same tokens
    for (int64_t t = (int64_t)blockIdx.x * G + wave / W; t < tokens; t += (int64_t)gridDim.x * G) {
        for (int j0 = 0; j0 < top_k; j0 += J) {
            const Rows<J> R = rows_of<J>(rows + t * top_k, j0, top_k, n_rows);
            float dot[J] = {};
            if (R.ok)
                for (int64_t u = part * 64 + lane; u < units; u += 64 * W) {
                    u32x4 v[J];
                    if (d_weights)
#pragma unroll
                        for (int j = 0; j < J; ++j) v[j] = ((const u32x4*)ys)[(int64_t)R.r[j] * units + u];
                    float g[U];
                    load_u<DT, U>(dy, t * units + u, g);
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        if (!(R.ok >> j & 1)) continue;
                        float f[U];
                        if (d_weights) {
                            unpack<ST, U>(v[j], f);
#pragma unroll
                            for (int i = 0; i < U; ++i) dot[j] = fmaf(g[i], f[i], dot[j]);
                        }
                        if (d_ys) {
                            const float w = weights ? weights[t * top_k + j0 + j] : 1.0f;
#pragma unroll
                            for (int i = 0; i < U; ++i) f[i] = g[i] * w;
                            store_u<ST, U>(d_ys, (int64_t)R.r[j] * units + u, f);
                        }
                    }
                }
            if (!d_weights) continue;
            float s = wave_sum8(dot);
            if constexpr (W > 1) {
                if ((lane & 7) == 0) red[wave][lane >> 3] = s;
                __syncthreads();
                s = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) s += red[w][lane >> 3];
                __syncthreads();
            }
            const int j = j0 + (lane >> 3);
            if (part == 0 && (lane & 7) == 0 && j < top_k) d_weights[t * top_k + j] = s;
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

// Workgroups (a multiple of 4) and pairs per workgroup of the two-launch sort.
int64_t sort_blocks(int64_t P, int64_t* per)
{
    int64_t n = ((P + kBlockPairs - 1) / kBlockPairs + 3) / 4 * 4;
    if (n > kMaxBlocks) n = kMaxBlocks;
    *per = n ? (P + n - 1) / n : 0;
    return n;
}

// Grid of a row kernel with runs of 64 V units, and log2 of the runs per workgroup.
dim3 row_grid(int64_t tokens, int64_t units, int V, int* lw)
{
    const int64_t runs = (units + 64 * V - 1) / (64 * V);
    *lw = runs <= 1 ? 0 : runs == 2 ? 1 : 2;
    return dim3(grid_of(tokens, 4 >> *lw), runs ? (unsigned)((runs + (1 << *lw) - 1) >> *lw) : 1);
}

template <int T>
void sort_in_two(const int32_t* experts, int64_t P, int E, int bits, int32_t* counts, int32_t* rows, int32_t* pairs,
                 int32_t* offsets, hipStream_t st)
{
    int64_t per;
    const unsigned n = (unsigned)sort_blocks(P, &per);
    const size_t lds = T / 64 * (E + 1) * 4;
    hipLaunchKernelGGL(k_sort_count<T>, dim3(n), dim3(T), lds, st, experts, P, per, E, counts);
    hipLaunchKernelGGL(k_sort_place<T>, dim3(n), dim3(T), lds, st, experts, P, per, E, bits, (const int32_t*)counts,
                       rows, pairs, offsets);
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
    *bytes = 0;
    if (P > kSmallPairs || (P > kFewPairs && n_experts > kSmallExperts))
        *bytes = (size_t)tq_align256(sort_blocks(P, &per) * (n_experts + 1) * 4);
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
    const int64_t units = copy ? width * size_of(x_type) / 16 : 0;
    const u32x4* xp = copy ? (const u32x4*)x : nullptr;
    const float* xsc = scales ? x_scale : nullptr;
    int lw;
    dim3 grid = row_grid(tokens, units, 1, &lw);
    if (P <= kFewPairs) {
        ++grid.x;
        const auto few = P <= 256 ? k_dispatch_few<4> : P <= 512 ? k_dispatch_few<8> : k_dispatch_few<kFewPairs / 64>;
        hipLaunchKernelGGL(few, grid, dim3(256), 0, st, experts, (int)tokens, top_k, n_experts, rows, pairs, offsets,
                           units, lw, xp, xsc, (u32x4*)xs, xs_scale);
        if ((s = tq_check_launch("tq_moe_dispatch"))) return s;
        return tq_ok();
    }
    if (need == 0) {
        hipLaunchKernelGGL(k_sort_one, dim3(1), dim3(kSortThreads), kSortThreads / 64 * (n_experts + 1) * 4, st,
                           experts, P, n_experts, bits, rows, pairs, offsets);
    } else {
        // 16 waves' counters of n_experts + 1 buckets within 64 KiB of LDS, or 8 waves'
        const auto sort = n_experts <= kSmallExperts ? sort_in_two<1024> : sort_in_two<512>;
        sort(experts, P, n_experts, bits, (int32_t*)workspace, rows, pairs, offsets, st);
    }
    if ((s = tq_check_launch("tq_moe_dispatch sort"))) return s;
    if (copy || scales) {
        hipLaunchKernelGGL(k_spread_rows, grid, dim3(256), 0, st, tokens, top_k, units, lw, rows, xp, xsc, (u32x4*)xs,
                           xs_scale);
        if ((s = tq_check_launch("tq_moe_dispatch rows"))) return s;
    }
    return tq_ok();
}

namespace {

template <int ST, int YT, int J, int V>
void launch_combine_as(int64_t tokens, int top_k, int64_t units, int64_t n_rows, const int32_t* rows,
                       const float* weights, const void* ys, void* y, hipStream_t st)
{
    int lw;
    const dim3 grid = row_grid(tokens, units, V, &lw);
    hipLaunchKernelGGL((k_combine<ST, YT, J, V>), grid, dim3(256), 0, st, tokens, top_k, units, lw, n_rows, rows, weights,
                       ys, y);
}

// 16 loads of 16 bytes in flight per lane: over the pairs, then along the row.
template <int ST, int YT>
void launch_combine(int64_t tokens, int top_k, int64_t width, int64_t n_rows, const int32_t* rows, const float* weights,
                    const void* ys, void* y, hipStream_t st)
{
    const int64_t units = width / unit_of<ST>();
    if (top_k == 1) launch_combine_as<ST, YT, 1, 4>(tokens, top_k, units, n_rows, rows, weights, ys, y, st);
    else if (top_k == 2) launch_combine_as<ST, YT, 2, 4>(tokens, top_k, units, n_rows, rows, weights, ys, y, st);
    else if (top_k <= 4) launch_combine_as<ST, YT, 4, 4>(tokens, top_k, units, n_rows, rows, weights, ys, y, st);
    else launch_combine_as<ST, YT, 8, 2>(tokens, top_k, units, n_rows, rows, weights, ys, y, st);
}

template <int DT, int ST>
void launch_grad(int64_t tokens, int top_k, int64_t width, int64_t n_rows, const int32_t* rows, const float* weights,
                 const void* dy, const void* ys, void* d_ys, float* d_weights, hipStream_t st)
{
    const int64_t units = width / unit_of<ST>();
    if (units <= 64)
        hipLaunchKernelGGL((k_combine_grad<DT, ST, 1>), dim3(grid_of(tokens, 4)), dim3(256), 0, st, tokens, top_k,
                           units, n_rows, rows, weights, dy, ys, d_ys, d_weights);
    else    // 4099 tokens, 8 rows of 2048 bf16: 57.9 us; with one wave per token and two units per lane 71 us
        hipLaunchKernelGGL((k_combine_grad<DT, ST, 4>), dim3(grid_of(tokens, 1)), dim3(256), 0, st, tokens, top_k,
                           units, n_rows, rows, weights, dy, ys, d_ys, d_weights);
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
    const Span in[] = {{rows, P * 4, "rows"}, {weights, P * 4, "weights"},
                       {ys, n_rows * width * size_of(ys_type), "ys"}};
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
    const Span in[] = {{rows, P * 4, "rows"}, {weights, P * 4, "weights"},
                       {dy, tokens * width * size_of(dy_type), "dy"},
                       {ys, d_weights ? n_rows * row : 0, "ys"}};
    if ((s = check_spans(out, in))) return s;
    auto* fn = dy_type == TQ_F32 ? (ys_type == TQ_F32 ? launch_grad<TQ_F32, TQ_F32> : launch_grad<TQ_F32, TQ_BF16>)
                                 : (ys_type == TQ_F32 ? launch_grad<TQ_BF16, TQ_F32> : launch_grad<TQ_BF16, TQ_BF16>);
    fn(tokens, top_k, width, n_rows, rows, weights, dy, ys, d_ys, d_weights, (hipStream_t)stream);
    if ((s = tq_check_launch("tq_moe_combine_grad"))) return s;
    return tq_ok();
}
