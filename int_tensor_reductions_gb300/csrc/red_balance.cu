// red_balance.cu -- balance loss of a router of experts, with the experts'
// counts and the gradient by the router's logits (red_balance).
//
// With n the tokens that take part and count_e the entries of their ids that
// name expert e,
//     share_e = count_e / (k n),  prob_e = mean over them of p_te,
//     loss = coef * E * sum_e share_e prob_e + z_coef * mean lse_t^2.
// The counts do not depend on the logits, and the gradient depends on the other
// tokens through the counts alone:
//     d loss / dp_te = c_e = coef E share_e / n,
// so that after the counts one pass reads the logits, writes the gradient and
// sums p.  Three kernels: counts (integer atomics: any order gives the same),
// rows, and a join of the CTAs' sums; one CTA does all three where tokens are
// few.  Bound by instructions: 65536 x 256 sigmoids take 33.0 us in f32 and 29.7 in
// bf16, half the bytes (softmax 31.7, 26.2; memory's share 19.9 and 10), and the rows' kernel 74%
// of the issue slots.  Few tokens are bound by latency.
#include "red_balance.cuh"
#include "red_groups.cuh"
#include "red_prims.cuh"

namespace red {
namespace {

// Workspace: counters of the experts and of the tokens (zero between calls), the number of
// tokens for the join, and the CTAs' sums: of p for each expert, of lse^2, of count_e p_te.
__device__ __forceinline__ unsigned *tokens_seen(const BalanceArgs &a) { return reinterpret_cast<unsigned *>(a.part); }
__device__ __forceinline__ float *sums_at(const BalanceArgs &a, int64_t cta)
{
    return a.part + 4 + cta * (a.experts + 2);
}

constexpr int COUNT_NT = 1024;

// Adds the ids' entries to the counters in shared memory: eight loads at a time, and
// what depends on them afterwards (one after the other they took 8 us of 500,000).
__device__ __forceinline__ void count_ids(const BalanceArgs &a, unsigned *counts, unsigned *tokens, int64_t first,
                                          int64_t step)
{
    constexpr int BATCH = 8;
    const int64_t entries = a.rows * a.k;
    unsigned mine = 0;
    for (int64_t i0 = first; i0 < entries; i0 += BATCH * step) {
        int64_t id[BATCH];
        unsigned takes = 0;
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int64_t i = i0 + b * step;
            const bool in = i < entries;
            id[b] = in ? a.ids[i] : -1;
            // (below 2^31 entries: 32-bit division)
            const unsigned row = (unsigned)i / (unsigned)a.k;
            if (in && (!a.live || a.live[row])) {
                takes |= 1u << b;
                mine += row * (unsigned)a.k == (unsigned)i;
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
            if ((takes >> b & 1) && id[b] >= 0 && id[b] < a.experts)
                atomicAdd(counts + id[b], 1u);
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (threadIdx.x % 32 == 0 && mine)
        atomicAdd(tokens, mine);
}

__global__ void __launch_bounds__(COUNT_NT) balance_count_kernel(const BalanceArgs a)
{
    // The rows kernel may come once what precedes this call is done: its first rows are
    // on their way while the ids are counted.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ unsigned counts[];  // experts, tokens
    for (int e = threadIdx.x; e <= a.experts; e += COUNT_NT)
        counts[e] = 0;
    __syncthreads();
    count_ids(a, counts, counts + a.experts, (int64_t)blockIdx.x * COUNT_NT + threadIdx.x, (int64_t)gridDim.x * COUNT_NT);
    __syncthreads();
    for (int e = threadIdx.x; e <= a.experts; e += COUNT_NT)
        if (counts[e])
            atomicAdd(a.tick + (e < a.experts ? e : RED_BALANCE_MAX_EXPERTS), counts[e]);
}

// A lane's share of the counts, and its sums over rows.
template <int N, int E>
struct RowSums {
    float c[N][E], p[N][E];
    float z, d;    // of lse^2, and of the tokens' sums of count_e p_te
    float unit;    // of count_e in the gradient
};

__device__ __forceinline__ bool takes_part(const BalanceArgs &a, int64_t r)
{
    return r < a.rows && (!a.live || a.live[r]);
}
__device__ __forceinline__ float tokens_of(unsigned n) { return (float)(n ? n : 1u); }

template <int LANES, int N, int E>
__device__ __forceinline__ void begin_sums(const BalanceArgs &a, RowSums<N, E> &s, const unsigned *counts, float n, int lane)
{
    s.unit = a.coef * a.grad_scale * (float)a.experts / ((float)a.k * n * n);
#pragma unroll
    for (int v = 0; v < N; ++v)
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int e = (v * LANES + lane) * E + k;
            s.c[v][k] = e < a.experts ? (float)counts[e] : 0.0f;
            s.p[v][k] = 0.0f;
        }
    s.z = s.d = 0.0f;
}

// The sigmoid of what balance_row keeps of it.
__device__ __forceinline__ bool negative(float e) { return __float_as_int(e) < 0; }
__device__ __forceinline__ float numerator(float e) { return negative(e) ? 1.0f + e : e; }

// One token's logits: its probabilities into the sums, its gradient to memory.
// `here`: there is such a token; a group without one goes along.
template <int DT, bool SIGMOID, int LANES, bool VEC, int N, int E>
__device__ __forceinline__ void balance_row(const BalanceArgs &a, const Raw (&raw)[N], RowSums<N, E> &s,
                                            GroupShared<LANES> &sh, int &turn, float z_unit, int64_t r, bool here,
                                            bool takes, int lane)
{
    float x[N][E];
    float top = NEG_INF;
#pragma unroll
    for (int v = 0; v < N; ++v) {
        const int i = (v * LANES + lane) * E;
        widen<DT>(raw[v], x[v]);
        if (i + E > a.experts) {
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (i + k >= a.experts)
                    x[v][k] = NEG_INF;
        }
        if (!SIGMOID) {
#pragma unroll
            for (int k = 0; k < E; ++k)
                top = Max()(top, x[v][k]);
        }
    }
    float off = 0.0f;  // (differences first: a row of the type's lowest value has no room for a product)
    // exponentials, or of a sigmoid and its complement the smaller one, negative where it is the complement: 1 - s of an s
    // near 1 has no digits (at a logit of 10 it was off by 5e-4, from 17 on it was 0, and so was the gradient)
    float e[N][E];
    if constexpr (!SIGMOID) {
        top = group_fold<LANES>(top, sh, turn, Max());
        off = top == NEG_INF ? 0.0f : top;
    }
    // sum of e and of e * c, for sum of p * c
    float2 sums = make_float2(0.0f, 0.0f);
    [[maybe_unused]] float keep = 1.0f;  // sigmoids: 0 where e is p's numerator alone, and the complement 1
#pragma unroll
    for (int v = 0; v < N; ++v)
#pragma unroll
        for (int k = 0; k < E; ++k) {
            float n;  // of p: its numerator
            if constexpr (SIGMOID) {
                const float u = ex2(-fabsf(x[v][k]) * LOG2E), r = __fdividef(1.0f, 1.0f + u);
                n = x[v][k] >= 0.0f ? r : u * r;
                e[v][k] = x[v][k] >= 0.0f ? -(u * r) : n;
            } else {
                n = e[v][k] = ex2((x[v][k] - off) * LOG2E);
            }
            sums.x += n;
            sums.y = fmaf(n, s.c[v][k], sums.y);
        }
    sums = group_sums<LANES>(sums, sh, turn);
    if constexpr (SIGMOID) {
        // Logits below -69 throughout: 1 + e^x is 1, and p the softmax, whose terms do not underflow.
        // Below -700 (a mask's lowest value, in 64 bits a sigmoid of 0) there are no probabilities.
        // (For all groups of a warp at once: the others' sums become what they were.)
        const bool low = sums.x < 1e-30f;
        if (__any_sync(0xffffffffu, low)) {
#pragma unroll
            for (int v = 0; v < N; ++v)
#pragma unroll
                for (int k = 0; k < E; ++k)
                    top = Max()(top, x[v][k]);
            top = group_fold<LANES>(top, sh, turn, Max());
            keep = low ? 0.0f : 1.0f;
            sums = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int v = 0; v < N; ++v)
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    if (low)
                        e[v][k] = top < -700.0f ? 0.0f : ex2((x[v][k] - top) * LOG2E);
                    const float n = numerator(e[v][k]);
                    sums.x += n;
                    sums.y = fmaf(n, s.c[v][k], sums.y);
                }
            sums = group_sums<LANES>(sums, sh, turn);
        }
    }
    float sum = sums.x;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // nothing but -inf: no probabilities
    float d = sums.y * inv;
    if (!takes) {  // (its results so far are not looked at: they may be NaN)
#pragma unroll
        for (int v = 0; v < N; ++v)
#pragma unroll
            for (int k = 0; k < E; ++k)
                x[v][k] = e[v][k] = 0.0f;
        sum = d = 0.0f;
    } else {
#pragma unroll
        for (int v = 0; v < N; ++v)
#pragma unroll
            for (int k = 0; k < E; ++k)
                x[v][k] = (SIGMOID ? numerator(e[v][k]) : e[v][k]) * inv;
    }
#pragma unroll
    for (int v = 0; v < N; ++v)
#pragma unroll
        for (int k = 0; k < E; ++k)
            s.p[v][k] += x[v][k];
    s.d += d;
    float by_lse = 0.0f;
    if constexpr (!SIGMOID) {
        const float lse = sum == 0.0f ? 0.0f : fmaf(log2f(sum), 0.6931471805599453f, off);
        s.z = fmaf(lse, lse, s.z);
        by_lse = z_unit * lse;
    }
    if (!a.dx)
        return;
    const float shift = by_lse - d * s.unit;
#pragma unroll
    for (int v = 0; v < N; ++v) {
        float g[E];
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const float p = x[v][k];
            g[k] = (SIGMOID ? p * (negative(e[v][k]) ? -e[v][k] : fmaf(-keep, e[v][k], 1.0f)) : p) *
                   fmaf(s.c[v][k], s.unit, shift);
        }
        store_unit<DT, VEC, LANES>(a.dx, r * a.ldd, (v * LANES + lane) * E, a.experts, here, g);
    }
}

// The groups' sums of a CTA in `meet` (a row of LANES * VECS * 8 per warp, or per
// CTA), ready for sum_of().
template <int LANES, int N, int E>
__device__ __forceinline__ void meet_sums(RowSums<N, E> &s, float *meet, float2 *meet_zd, int lane)
{
    constexpr int WIDTH = LANES * N * E;
    float *const row = LANES > 32 ? meet : meet + threadIdx.x / 32 * WIDTH;
    if constexpr (LANES < 32) {
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
#pragma unroll
            for (int v = 0; v < N; ++v)
#pragma unroll
                for (int k = 0; k < E; ++k)
                    s.p[v][k] += __shfl_xor_sync(0xffffffffu, s.p[v][k], o);
            s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
            s.d += __shfl_xor_sync(0xffffffffu, s.d, o);
        }
    }
    if (LANES > 32 || threadIdx.x % 32 < LANES) {
#pragma unroll
        for (int v = 0; v < N; ++v)
#pragma unroll
            for (int k = 0; k < E; ++k)
                row[(v * LANES + lane) * E + k] = s.p[v][k];
    }
    if (LANES > 32 ? threadIdx.x == 0 : threadIdx.x % 32 == 0)
        meet_zd[LANES > 32 ? 0 : threadIdx.x / 32] = make_float2(s.z, s.d);
    __syncthreads();
}
template <int LANES, int VECS, int NT>
__device__ __forceinline__ float sum_of(const float *meet, int e)
{
    float p = meet[e];
    if constexpr (LANES <= 32) {
#pragma unroll
        for (int w = 1; w < NT / 32; ++w)
            p += meet[w * LANES * VECS * 8 + e];
    }
    return p;
}
template <int LANES, int NT>
__device__ __forceinline__ float2 sum_of_zd(const float2 *meet_zd)
{
    float2 s = meet_zd[0];
    if constexpr (LANES <= 32) {
#pragma unroll
        for (int w = 1; w < NT / 32; ++w) {
            s.x += meet_zd[w].x;
            s.y += meet_zd[w].y;
        }
    }
    return s;
}

template <int DT, bool SIGMOID, int LANES, int VECS, bool VEC>
__global__ void __launch_bounds__(GROUP_CTA<LANES>) balance_rows_kernel(const BalanceArgs a)
{
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES, N = UNITS<DT, VECS>, E = UNIT<DT>;
    __shared__ GroupShared<LANES> sh;
    __shared__ float meet[(LANES > 32 ? 1 : NT / 32) * LANES * VECS * 8];
    __shared__ float2 meet_zd[NT / 32];
    using Rows = Ring<DT, VEC, LANES, UNITS<DT, VECS>, 1>;
    extern __shared__ __align__(16) unsigned char ring[];
    const Rows rows = {ring, 1};
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const int64_t step = (int64_t)gridDim.x * GROUPS, first = (int64_t)blockIdx.x * GROUPS + group;
    auto fetch = [&](int64_t r, int to) {
        if (r < a.rows)  // (one that is out is fetched, too: what says so is not known yet)
            rows.fetch(to, 0, a.x, r * a.ldx, lane, a.experts);
        fetch_commit();
    };
#pragma unroll
    for (int k = 0; k < Rows::STAGES - 1; ++k)
        fetch(first + k * step, k);
    pdl_enter();  // (x is the caller's, complete before the counts began)
    const float n = tokens_of(a.tick[RED_BALANCE_MAX_EXPERTS]);
    RowSums<N, E> s;
    begin_sums<LANES>(a, s, a.tick, n, lane);
    const float z_unit = 2.0f * a.z_coef * a.grad_scale / n;
    int turn = 0, stage = 0;
    bool next_takes = takes_part(a, first);
    for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < a.rows; r0 += step) {
        const int64_t r = r0 + group;
        const bool takes = next_takes;
        next_takes = takes_part(a, r + step);
        Raw raw[N];
        fetch(r + (Rows::STAGES - 1) * step, (stage + Rows::STAGES - 1) % Rows::STAGES);
        fetch_wait<Rows::STAGES - 1>();
#pragma unroll
        for (int v = 0; v < N; ++v)
            raw[v] = rows.take(stage, 0, v, a.x, r * a.ldx, lane, a.experts);
        stage = (stage + 1) % Rows::STAGES;
        balance_row<DT, SIGMOID, LANES, VEC>(a, raw, s, sh, turn, z_unit, r, r < a.rows, takes, lane);
    }
    meet_sums<LANES>(s, meet, meet_zd, lane);
    float *const part = sums_at(a, blockIdx.x);
    for (int e = threadIdx.x; e < a.experts; e += NT)
        part[e] = sum_of<LANES, VECS, NT>(meet, e);
    if (threadIdx.x == 0) {
        const float2 zd = sum_of_zd<LANES, NT>(meet_zd);
        part[a.experts] = zd.x;
        part[a.experts + 1] = zd.y;
        if (blockIdx.x == 0)
            *tokens_seen(a) = a.tick[RED_BALANCE_MAX_EXPERTS];
    }
}

// loss, its two parts and the tokens, from sum_e count_e * (sum of p_e) and the sum of lse^2.
__device__ __forceinline__ void write_stats(const BalanceArgs &a, unsigned tokens, float dot, float z)
{
    const float n = tokens_of(tokens);
    const float balance = dot * (float)a.experts / ((float)a.k * n * n);
    z /= n;
    a.stats[0] = a.z_coef == 0.0f ? a.coef * balance : fmaf(a.coef, balance, a.z_coef * z);  // (z may be infinite)
    a.stats[1] = balance;
    a.stats[2] = z;
    a.stats[3] = (float)tokens;
}

// Eight columns of the CTAs' sums per CTA by 128 lanes of CTAs.  Each clears the counters
// that it has read; that of the tokens has been read by then, and is `seen` besides.
constexpr int JOIN_NT = 1024, JOIN_WIDTH = 8;
__global__ void __launch_bounds__(JOIN_NT) balance_join_kernel(const BalanceArgs a, int parts)
{
    pdl_enter();
    __shared__ float sums[JOIN_NT / 32][JOIN_WIDTH];
    __shared__ float zd[2];
    // the last two columns are of one CTA
    const int col = threadIdx.x % JOIN_WIDTH, e = a.experts + 2 - (blockIdx.x + 1) * JOIN_WIDTH + col;
    const unsigned tokens = *tokens_seen(a);
    float p = 0.0f;
    if (e >= 0) {
#pragma unroll 8
        for (int i = threadIdx.x / JOIN_WIDTH; i < parts; i += JOIN_NT / JOIN_WIDTH)
            p += sums_at(a, i)[e];
    }
    for (int o = 16; o >= JOIN_WIDTH; o >>= 1)
        p += __shfl_xor_sync(0xffffffffu, p, o);
    if (threadIdx.x % 32 < JOIN_WIDTH)
        sums[threadIdx.x / 32][col] = p;
    __syncthreads();
    if (threadIdx.x < JOIN_WIDTH && e >= 0) {
        p = 0.0f;
#pragma unroll
        for (int w = 0; w < JOIN_NT / 32; ++w)
            p += sums[w][col];
        if (e < a.experts) {
            a.counts[e] = a.tick[e];
            a.tick[e] = 0;
            a.prob[e] = p / tokens_of(tokens);
        } else {
            zd[e - a.experts] = p;
        }
    }
    if (blockIdx.x == 0) {
        __syncthreads();
        if (threadIdx.x == 0) {
            a.tick[RED_BALANCE_MAX_EXPERTS] = 0;
            write_stats(a, tokens, zd[1], zd[0]);
        }
    }
}

// Few tokens: the CTAs of one cluster count, pass over the rows and join, through
// shared memory.  us, softmax f32 k 6: 257 x 64 8.4 with one
// CTA of 1024 threads, 6.9 with a cluster; 1000 x 64 14.8, 7.6; 4000 x 64 14.4 with a cluster, 11.7 with the three
// kernels below.
constexpr int FEW_THREADS = 512;
constexpr int FEW_EXPERTS = 256;
constexpr int FEW_CLUSTER = 8;

template <int DT, bool SIGMOID, int LANES, bool VEC>
__global__ void __launch_bounds__(FEW_THREADS) balance_few_kernel(const BalanceArgs a)
{
    pdl_enter();
    constexpr int GROUPS = FEW_THREADS / LANES, N = UNITS<DT, 1>, E = UNIT<DT>;
    __shared__ GroupShared<LANES> sh;
    __shared__ float meet[FEW_THREADS / 32 * LANES * 8];
    __shared__ float2 meet_zd[FEW_THREADS / 32];
    __shared__ float share[FEW_EXPERTS + 2], sums[FEW_EXPERTS + 2];
    __shared__ unsigned mine[FEW_EXPERTS + 1], counts[FEW_EXPERTS + 1];  // experts, tokens
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const int ctas = cluster_size(), rank = cluster_rank();
    const int64_t step = ctas * GROUPS, first = rank * GROUPS + group;
    for (int e = threadIdx.x; e <= FEW_EXPERTS; e += FEW_THREADS)
        mine[e] = 0;
    // the first token's logits are on their way while the ids are counted, the next one's while one is at work
    Raw next[N];
    bool next_takes = takes_part(a, first);
    load_row<DT, VEC, LANES>(next, a.x, next_takes ? first * a.ldx : 0, lane, next_takes ? a.experts : 0);
    __syncthreads();
    count_ids(a, mine, mine + FEW_EXPERTS, rank * FEW_THREADS + threadIdx.x, ctas * FEW_THREADS);
    __syncthreads();
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    }
    if (threadIdx.x <= FEW_EXPERTS) {
        unsigned n = 0;
        for (int c = 0; c < ctas; ++c)
            n += *in_cta(mine + threadIdx.x, c);
        counts[threadIdx.x] = n;
    }
    __syncthreads();
    const unsigned tokens = counts[FEW_EXPERTS];
    const float n = tokens_of(tokens);
    RowSums<N, E> s;
    begin_sums<LANES>(a, s, counts, n, lane);
    const float z_unit = 2.0f * a.z_coef * a.grad_scale / n;
    int turn = 0;
    for (int64_t r0 = rank * GROUPS; r0 < a.rows; r0 += step) {
        const int64_t r = r0 + group;
        Raw raw[N];
#pragma unroll
        for (int v = 0; v < N; ++v)
            raw[v] = next[v];
        const bool takes = next_takes;
        next_takes = takes_part(a, r + step);
        load_row<DT, VEC, LANES>(next, a.x, next_takes ? (r + step) * a.ldx : 0, lane, next_takes ? a.experts : 0);
        balance_row<DT, SIGMOID, LANES, VEC>(a, raw, s, sh, turn, z_unit, r, r < a.rows, takes, lane);
    }
    meet_sums<LANES>(s, meet, meet_zd, lane);
    if (threadIdx.x < a.experts)
        share[threadIdx.x] = sum_of<LANES, 1, FEW_THREADS>(meet, threadIdx.x);
    if (threadIdx.x == 0) {
        const float2 zd = sum_of_zd<LANES, FEW_THREADS>(meet_zd);
        share[a.experts] = zd.x;
        share[a.experts + 1] = zd.y;
    }
    // every sum to the first CTA
    float *const all = in_cta(sums, 0);
    cluster_sums(share, a.experts + 2, [&](int e, float sum) { all[e] = sum; });
    if (rank != 0)
        return;
    __syncthreads();
    if (threadIdx.x < a.experts) {
        a.counts[threadIdx.x] = counts[threadIdx.x];
        a.prob[threadIdx.x] = sums[threadIdx.x] / n;
    }
    if (threadIdx.x == 0)
        write_stats(a, tokens, sums[a.experts + 1], sums[a.experts]);
}

// One cluster does all of it up to this many logits; a CTA of it has at least this many.
constexpr int64_t FEW_LOGITS = 1 << 17, FEW_PER_CTA = 1 << 12;

template <int DT, bool SIGMOID, int LANES, bool VEC>
int launch_few(const BalanceArgs &a, cudaStream_t s)
{
    unsigned cluster = 1;
    while (cluster < FEW_CLUSTER && cluster * FEW_PER_CTA < a.rows * a.experts)
        cluster *= 2;
    count_launches(1);
    return cuda_fail(launch_pdl_smem(balance_few_kernel<DT, SIGMOID, LANES, VEC>, cluster, FEW_THREADS, 0, cluster, s, a),
                     "balance_few");
}

template <int DT, bool SIGMOID, int LANES, int VECS, bool VEC>
int launch_rows(BalanceArgs &a, cudaStream_t s)
{
    static Resident cache;
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES;
    DeviceInfo di;
    int st = device_info(&di);
    Workspace ws;
    if (st == RED_OK)
        st = get_workspace(&ws);
    constexpr size_t SMEM = Ring<DT, VEC, LANES, UNITS<DT, VECS>, 1>::bytes(1);
    unsigned grid = 1;
    auto *const kernel = balance_rows_kernel<DT, SIGMOID, LANES, VECS, VEC>;
    if (st == RED_OK)
        st = resident_grid(kernel, cache, NT, SMEM, SMEM, (a.rows + GROUPS - 1) / GROUPS,
                           (int64_t)(WS_PART_ELEMS / (size_t)(a.experts + 2)) - 1, &grid);
    if (st != RED_OK)
        return st;
    a.tick = ws.tick;
    a.part = static_cast<float *>(ws.part);
    const int64_t per = 4 * COUNT_NT, want = (a.rows * a.k + per - 1) / per;
    st = cuda_fail(launch_pdl_dynamic(balance_count_kernel, dim3((unsigned)(want < di.sms ? want : di.sms)), dim3(COUNT_NT),
                                      (size_t)(a.experts + 1) * sizeof(unsigned), s, a),
                   "balance_count");
    if (st == RED_OK)
        st = cuda_fail(launch_pdl_dynamic(kernel, dim3(grid), dim3(NT), SMEM, s, a),
                       "balance_rows");
    if (st == RED_OK)
        st = cuda_fail(launch_pdl(balance_join_kernel, dim3((unsigned)((a.experts + 1) / JOIN_WIDTH + 1)), dim3(JOIN_NT), s, a,
                                  (int)grid),
                       "balance_join");
    if (st == RED_OK)
        count_launches(3);
    else  // the next call finds the counters as they were
        cudaMemsetAsync(a.tick, 0, (RED_BALANCE_MAX_EXPERTS + 1) * sizeof(unsigned), s);
    return st;
}

template <int DT, bool SIGMOID>
int launch_typed_balance(BalanceArgs &a, cudaStream_t s)
{
    const int elem = DT == RED_F32 ? 4 : 2;
    const bool vec = aligned_rows(a.x, a.ldx, a.rows, elem) && aligned_rows(a.dx, a.ldd, a.rows, elem);
    return with_group((a.experts + 7) / 8, [&](auto lanes, auto vecs) {
        constexpr int L = decltype(lanes)::value, V = decltype(vecs)::value;
        if constexpr (V == 1) {
            if (a.rows * a.experts <= FEW_LOGITS)
                return vec ? launch_few<DT, SIGMOID, L, true>(a, s) : launch_few<DT, SIGMOID, L, false>(a, s);
        }
        // Two rows of 129 to 256 experts to a warp: what is done once per row is done for both (us, one / two:
        // 65536 x 256 f32 33.6 / 32.6, bf16 30.9 / 28.8, 30000 x 201 f32 26.4 / 24.7; with four rows of 65 to 128
        // for two, 65536 x 128 21.9 / 21.3, but 2000 x 100 8.3 / 8.9).
        constexpr int RL = V == 1 && L == 32 ? 16 : L, RV = V == 1 && L == 32 ? 2 : V;
        if constexpr (L * V * 8 <= RED_BALANCE_MAX_EXPERTS)
            return vec ? launch_rows<DT, SIGMOID, RL, RV, true>(a, s) : launch_rows<DT, SIGMOID, RL, RV, false>(a, s);
        else
            return fail(RED_EINVAL, "red_balance: too many experts");
    });
}

}  // namespace

int launch_balance(int dtype, BalanceArgs a, int kind, cudaStream_t s)
{
    const bool sigmoid = kind == RED_BALANCE_SIGMOID;
    switch (dtype) {
    case RED_F32: return sigmoid ? launch_typed_balance<RED_F32, true>(a, s) : launch_typed_balance<RED_F32, false>(a, s);
    case RED_F16: return sigmoid ? launch_typed_balance<RED_F16, true>(a, s) : launch_typed_balance<RED_F16, false>(a, s);
    default: return sigmoid ? launch_typed_balance<RED_BF16, true>(a, s) : launch_typed_balance<RED_BF16, false>(a, s);
    }
}

}  // namespace red
