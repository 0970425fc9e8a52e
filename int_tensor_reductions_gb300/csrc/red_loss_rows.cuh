// red_loss_rows.cuh -- the row kernel of the losses over logits: one pass
// over memory, the logits of a row held in shared memory between its
// statistics and its gradient.
//
// What bounds it is DRAM: each live row is read once and each row of the
// gradient written once (a multiply-add, an exponential and two conversions
// per element and pass are within the SM's rates, if little else is issued
// beside them).  So the kernel's work is to keep loads in flight all the time
// and the arithmetic warps free of everything else.  Persistent CTAs take
// rows from a counter.  A loader thread streams the rows into a ring of slots
// in shared memory with bulk copies: a row's slots stay until the gradient
// pass has read them, and each slot that this pass frees is filled at once
// with the next of the rows ahead.  A row longer than the ring drops its
// first batches after the statistics and has them fetched again for the
// gradient (from L2: they are a few microseconds old).
//
// A scheduler warp takes rows, reads their scalars (target, weight), writes
// zeros over the gradient of rows out of the loss and hands the others on
// through a queue; a writer warp joins a row's statistics, gives the other
// warps the coefficients of its gradient and writes its loss; for the
// distillation teacher warps do that, and read the rows' lists of teacher
// entries.
#pragma once

#include <type_traits>

#include "red_internal.h"
#include "red_loss.cuh"
#include "red_prims.cuh"

namespace red {

// ------------------------------------------------------- vectors of logits

template <int DT>
constexpr int VEC_ELEMS = DT == RED_F32 ? 4 : 8;  // in 16 bytes

// Two floats in one 64-bit register pair, the operand of Blackwell's packed
// fp32 instructions.
using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pack2(float a, float b)
{
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 unpack2(f32x2 v)
{
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f32x2 exp2_2(f32x2 v)
{
    const float2 f = unpack2(v);
    return pack2(ex2(f.x), ex2(f.y));
}

// Pair i of a vector, widened.
template <int DT>
__device__ __forceinline__ f32x2 vec_pair(const uint4 &v, int i)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (DT == RED_F32) {
        return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else if constexpr (DT == RED_BF16) {
        return pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
        __half2 h;
        memcpy(&h, &w[i], 4);
        const float2 f = __half22float2(h);
        return pack2(f.x, f.y);
    }
}

// Largest element of a vector; NaN elements are passed over.
template <int DT>
__device__ __forceinline__ float vec_max(const uint4 &v)
{
    if constexpr (DT == RED_F32) {
        return fmaxf(max3f(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z)), __uint_as_float(v.w));
    } else if constexpr (DT == RED_BF16) {
        __nv_bfloat162 h[4];
        memcpy(h, &v, 16);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        __half2 h[4];
        memcpy(h, &v, 16);
        const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
}

template <int DT>
__device__ __forceinline__ uint4 vec_pack(const f32x2 (&f)[VEC_ELEMS<DT> / 2])
{
    uint4 v;
    if constexpr (DT == RED_F32) {
        memcpy(&v, f, 16);
    } else if constexpr (DT == RED_BF16) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = __float22bfloat162_rn(unpack2(f[i]));
        memcpy(&v, h, 16);
    } else {
        __half2 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = __float22half2_rn(unpack2(f[i]));
        memcpy(&v, h, 16);
    }
    return v;
}

// Running statistics of one thread; the sum in two lanes.
struct SoftRun {
    float m, m2;  // m2 = m * s2, rounded
    f32x2 l;

    __device__ __forceinline__ void init(float top, float s2)
    {
        m = top;
        m2 = __fmul_rn(top, s2);
        l = pack2(0.0f, 0.0f);
    }
    __device__ __forceinline__ void raise(float to, float s2)
    {
        to = fmaxf(m, to);
        const float t2 = __fmul_rn(to, s2);
        const float f = soft_factor(m, m2, to, t2, s2);
        l = mul2(l, pack2(f, f));
        m = to;
        m2 = t2;
    }
    // n vectors, none of whose elements is above m
    template <int DT, int N>
    __device__ __forceinline__ void add(const uint4 (&v)[N], float s2)
    {
        if (is_near(m2)) {
            const f32x2 a = pack2(s2, s2), b = pack2(-m2, -m2);
#pragma unroll
            for (int u = 0; u < N; ++u)
                add_near<DT>(v[u], a, b);
        } else {
#pragma unroll
            for (int u = 0; u < N; ++u)
                l = far_sum<DT>(v[u], m, s2, l);
        }
    }
    template <int DT>
    __device__ __forceinline__ void add_near(const uint4 &v, f32x2 a, f32x2 b)
    {
#pragma unroll
        for (int i = 0; i < VEC_ELEMS<DT> / 2; ++i)
            l = add2(l, exp2_2(fma2(vec_pair<DT>(v, i), a, b)));
    }
    __device__ __forceinline__ void add(float x, float s2) { l = add2(l, pack2(ex2(term(x, m, m2, s2)), 0.0f)); }
    // exponent of one logit under the maximum m, near or far
    static __device__ __forceinline__ float term(float x, float m, float m2, float s2)
    {
        // (nothing finite yet: -inf is no term, and a NaN is one)
        return is_near(m2) ? fmaf(x, s2, -m2) : (m == NEG_INF ? x : (x - m) * s2);
    }
    template <int DT>
    static __device__ __noinline__ f32x2 far_sum(uint4 v, float m, float s2, f32x2 l)
    {
        const float m2 = __fmul_rn(m, s2);
        for (int i = 0; i < VEC_ELEMS<DT> / 2; ++i) {
            const float2 x = unpack2(vec_pair<DT>(v, i));
            l = add2(l, pack2(ex2(term(x.x, m, m2, s2)), ex2(term(x.y, m, m2, s2))));
        }
        return l;
    }
    __device__ __forceinline__ SoftStat stat() const
    {
        const float2 f = unpack2(l);
        return SoftStat{m, f.x + f.y};
    }
};

// 16 bytes into shared memory, and the wait for all that the thread asked for.
__device__ __forceinline__ void async_load16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The gradient of one vector of logits whose first column is j0.
template <int DT, bool FAR_ROW = false>
__device__ __forceinline__ uint4 vec_grad(const uint4 &v, const RowGrad &g, int j0)
{
    constexpr int E = VEC_ELEMS<DT>;
    const f32x2 a = pack2(g.fa, g.fa), b = pack2(g.fb, g.fb), m = pack2(g.mul, g.mul);
    f32x2 o[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        f32x2 t = fma2(vec_pair<DT>(v, i), a, b);
        if (FAR_ROW)
            t = mul2(t, pack2(g.fc, g.fc));
        o[i] = mul2(exp2_2(t), m);
    }
    const unsigned at = (unsigned)(g.y - j0);
    if (at < (unsigned)E) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            o[i] = add2(o[i], pack2(at == 2 * i ? g.cy : 0.0f, at == 2 * i + 1 ? g.cy : 0.0f));
    }
    return vec_pack<DT>(o);
}

template <int DT>
__device__ __forceinline__ float elem_grad(float x, const RowGrad &g, int j)
{
    return g.mul * ex2(fmaf(x, g.fa, g.fb) * g.fc) + (j == g.y ? g.cy : 0.0f);
}

// A vector to the gradient: 16 bytes at once where the address allows.
template <int DT>
__device__ __forceinline__ void store_vec(void *p, const uint4 &v, bool aligned)
{
    if (aligned) {
        *static_cast<uint4 *>(p) = v;
        return;
    }
    constexpr int E = VEC_ELEMS<DT>;
    typename Elem<DT>::T t[E];
    memcpy(t, &v, 16);
#pragma unroll
    for (int i = 0; i < E; ++i)
        static_cast<typename Elem<DT>::T *>(p)[i] = t[i];
}

// A vector of NaN: the word 0x7fc07fc0 is one in each of the types.
__device__ __forceinline__ uint4 nan_vec()
{
    return make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
}

// Elements of p[0, len) before its first 16-byte boundary, at most len.
template <int DT>
__device__ __forceinline__ int head_elems(const void *p, int len)
{
    const int h = (int)((16u - (unsigned)((uintptr_t)p & 15u)) & 15u) / (int)sizeof(typename Elem<DT>::T);
    return h < len ? h : len;
}

// Zeros over one row of the gradient, by threads tid of nt.
template <int DT>
__device__ __forceinline__ void zero_row(typename Elem<DT>::T *g, int len, int tid, int nt)
{
    constexpr int E = VEC_ELEMS<DT>;
    const int h = head_elems<DT>(g, len), nvec = (len - h) / E;
    for (int i = tid; i < nvec; i += nt)
        reinterpret_cast<uint4 *>(g + h)[i] = make_uint4(0, 0, 0, 0);
    if (tid < h)
        g[tid] = 0;
    for (int j = h + nvec * E + tid; j < len; j += nt)
        g[j] = 0;
}

// --------------------------------------------------------------- pipeline

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t *bar, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

// No wait is without end.  One that runs out, after `limit` tries in vain (0:
// after 20 s, which takes a hardware fault), marks the CTA as failed; what it
// has not written by then becomes NaN.
struct Patience {
    unsigned limit;
    unsigned tries = 0;
    uint64_t since = 0;

    __device__ __forceinline__ explicit Patience(unsigned n) : limit(n) {}
    static __device__ __forceinline__ uint64_t now()
    {
        uint64_t t;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        return t;
    }
    // After a try in vain: whether to give up.
    __device__ __forceinline__ bool spent(volatile int *failed)
    {
        ++tries;
        if (limit != 0) {
            if (tries < limit && !*failed)
                return false;
        } else {
            if (tries % 256 != 0)
                return false;
            if (tries == 256)
                since = now();
            if (!*failed && now() - since < 20000000000ull)
                return false;
        }
        *failed = 1;
        return true;
    }
};

// Whether the phase was over before the wait ran out.
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile int *failed, unsigned limit)
{
    if (mbar_try(bar, parity))
        return true;
    Patience patience(limit);
    while (!mbar_try(bar, parity))
        if (patience.spent(failed))
            return false;
    return true;
}

// ---- clusters

__device__ __forceinline__ int cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}
__device__ __forceinline__ int cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return (int)r;
}
// The same shared variable in CTA `rank` of the cluster.
template <class V>
__device__ __forceinline__ V *in_cta(V *p, int rank)
{
    uint64_t d;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(d) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<V *>(d);
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// `bytes` (a multiple of 16) from src to shared memory; both 16-byte aligned.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

// `bytes` (a multiple of 16) from shared memory to dst, in this thread's
// current bulk group.
__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)),
                 "r"(bytes)
                 : "memory");
}

constexpr int ZERO_BYTES = 4096;

// Zeros over one row of the gradient, by a warp: bulk stores from a block of
// zeros in shared memory, on their way while the CTA goes on.
template <int DT>
__device__ __forceinline__ void zero_row_bulk(typename Elem<DT>::T *g, int len, const void *zeros)
{
    constexpr int E = VEC_ELEMS<DT>;
    const int lane = threadIdx.x & 31;
    const int h = head_elems<DT>(g, len), nvec = (len - h) / E;
    if (lane == 0) {
        constexpr int STEP = ZERO_BYTES / 16;
        for (int v = 0; v < nvec; v += STEP)
            bulk_store(g + h + (int64_t)v * E, zeros, (uint32_t)min(STEP, nvec - v) * 16u);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    if (lane < h)
        g[lane] = 0;
    if (h + nvec * E + lane < len)
        g[h + nvec * E + lane] = 0;
}
__device__ __forceinline__ void bulk_stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

constexpr int ROW_Q = 32;      // entries of the row queue
constexpr int ROW_MAX_SLOTS = 32;
constexpr int TEACHERS = 4;    // teacher warps: each has the time of this many rows for one list

// Shared memory of the row kernel behind the slots.
template <int NW>
struct RowShared {
    RowEntry queue[ROW_Q];
    SoftStat part[2][NW];  // statistics of row i's warps in part[i % 2]
    RowGrad grad;          // of the row at hand
    uint64_t full[ROW_MAX_SLOTS], empty[ROW_MAX_SLOTS];
    alignas(16) unsigned char zeros[ZERO_BYTES];
    int published;  // entries written to the queue
    int failed;     // a wait ran out
};

template <class OP>
constexpr int SERVICE_WARPS = 2 + (OP::TEACHER ? TEACHERS : OP::STATS);  // scheduler, loader, teachers or writer

__device__ __forceinline__ void bar_sync(int id, int n)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int n)
{
    __threadfence_block();
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// NT consumer threads and the service warps; `slots` batches of U * NT
// vectors in shared memory.  next: the row counter and the count of finished
// CTAs, both zero before and after.  limit: see Patience.
//
// The queue: entry i, a row of the loss, is in slot i % ROW_Q, and entries up to
// i + 1 + ahead can be read after row i is `given`.  The scheduler takes
// `group` rows at a time, when they are needed and not before: a row that
// waits in one CTA's queue at the end is one that another, idle by then, could
// have had (with the next rows always on their way: policy 8192 x 65536 bf16
// 300 us instead of 290).
template <int DT, class OP, int NT, int U>
__global__ void __launch_bounds__(NT + 32 * SERVICE_WARPS<OP>)
row_kernel(LogitRows a, OP op, unsigned *next, int slots, int group, int ahead, int teacher_k, unsigned limit)
{
    using T = typename Elem<DT>::T;
    constexpr int E = VEC_ELEMS<DT>, NW = NT / 32;
    static_assert((NW & (NW - 1)) == 0 && NW <= 32, "the join of the warps' statistics");
    extern __shared__ __align__(16) unsigned char smem[];
    uint4 *const ring = reinterpret_cast<uint4 *>(smem);
    using Shared = RowShared<NW>;
    Shared &sh = *reinterpret_cast<Shared *>(ring + slots * U * NT);
    unsigned char *const lists = reinterpret_cast<unsigned char *>(&sh + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float s2 = a.s2;
    pdl_enter();

    for (int i = tid; i < ZERO_BYTES / 16; i += blockDim.x)
        reinterpret_cast<uint4 *>(sh.zeros)[i] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (tid == 0) {
        for (int i = 0; i < slots; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], NW);
        }
        sh.published = 0;
        sh.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    volatile int *const failed = &sh.failed;
    volatile int *const published = &sh.published;

    // Named barriers.  Per row i, and for the distillation per teacher warp w =
    // i % TEACHERS: `summed`, the consumers' statistics are there (the writer, or
    // the teacher, waits); `given`, the gradient's coefficients and the next
    // entries are there (all wait, so that none reads an entry too early);
    // `done`, the row's gradient is written (its teacher waits).
    // The loader runs ahead by the slots alone.
    auto summed = [](int i) { return OP::TEACHER ? 1 + i % TEACHERS : 1; };
    auto given = [](int i) { return OP::TEACHER ? 1 + TEACHERS + i % TEACHERS : 2; };
    auto done = [](int i) { return 1 + 2 * TEACHERS + i % TEACHERS; };
    constexpr int GIVEN = NT + 32 + 32 * OP::STATS;  // threads of `given`
    // The first entries are there.
    auto first_barrier = [&]() { bar_sync(15, NT + 32 * (SERVICE_WARPS<OP> - 1)); };
    // Batches of a row of nvec vectors, and how many of them are fetched twice.
    auto batches = [](int nvec) { return (nvec + U * NT - 1) / (U * NT); };
    auto twice = [&](int nb) { return OP::STATS && a.dx && nb > slots ? nb - slots : 0; };
    // By the writer, or row i's teacher, between the consumers' statistics and
    // their gradient pass; the statistics.
    auto give_row = [&](int i, const RowEntry &e, float mass) {
        bar_sync(summed(i), NT + 32);
        // Copies of the NW parts throughout the warp, joined in log2(NW) levels.
        // They are read before `given`: the consumers write the same buffer for
        // row i + 2, and that only waits for row i + 1 to be given, which for the
        // distillation another warp does.
        const SoftStat part = sh.part[i % 2][lane % NW];
        if (!a.dx)
            bar_sync(given(i), GIVEN);
        SoftStat w = soft_warp<NW>(part, s2);
        if (*failed)
            w.l = __int_as_float(0x7fc00000);
        const RowStat t = row_stat(a, w);
        if (a.dx) {
            const RowGrad g = op.template grad<DT>(a, e, t, mass);
            if (lane == 0)
                sh.grad = g;
            __syncwarp();
            bar_sync(given(i), GIVEN);
        }
        return t;
    };

    if (warp == NW) {
        // ---- scheduler
        int count = 0;       // entries published
        bool ended = false;  // and the last of them is the end
        bool first = true;   // the first rows are fixed, the rest come from the counter
        RowEntry got;        // an entry in each of the first `group` lanes,
        int64_t base = 0;    // rows base, base + 1, ... (as the loss counts them)
        auto load = [&]() {
            unsigned t = 0;
            if (!first && lane == 0)
                t = atomicAdd(next, (unsigned)group);
            t = __shfl_sync(0xffffffffu, t, 0);
            base = first ? (int64_t)blockIdx.x * group : (int64_t)gridDim.x * group + t;
            first = false;
            if (lane < group && base + lane < a.rows)
                op.load(base + lane, got);
        };
        auto publish = [&]() {
            const bool in = lane < group && base + lane < a.rows;
            if (in)
                op.settle(a, got);
            const bool live = in && got.state == ROW_LIVE;
            const unsigned lives = __ballot_sync(0xffffffffu, live);
            unsigned outs = __ballot_sync(0xffffffffu, in && !live);
            ended = base >= a.rows;
            if (live)
                sh.queue[(count + __popc(lives & ((1u << lane) - 1u))) % ROW_Q] = got;
            if (ended && lane == 0)
                sh.queue[count % ROW_Q].state = ROW_END;
            count += __popc(lives) + ended;
            __syncwarp();
            __threadfence_block();
            if (lane == 0)
                *published = count;
            if (in && !live)
                op.skip(got.r);
            for (; a.dx && outs; outs &= outs - 1) {
                const int64_t r = __shfl_sync(0xffffffffu, got.r, __ffs(outs) - 1);
                zero_row_bulk<DT>(static_cast<T *>(a.dx) + r * a.ldd, a.len, sh.zeros);
            }
        };
        auto want = [&](int upto) {
            while (!ended && count < upto) {
                load();
                publish();
            }
        };
        want(1 + ahead);
        first_barrier();
        for (int i = 0; sh.queue[i % ROW_Q].state != ROW_END; ++i) {
            want(i + 2 + ahead);
            bar_sync(given(i), GIVEN);
        }
        if (lane == 0)
            bulk_stores_done();
        // the last to finish leaves the counters as they were
        if (lane == 0) {
            __threadfence();
            if (atomicAdd(next + 1, 1u) == gridDim.x - 1) {
                next[0] = 0;
                next[1] = 0;
            }
        }
    } else if (warp == NW + 1 && lane == 0) {
        // ---- loader
        int slot = 0;
        uint32_t parity = 1;  // a fresh slot is empty
        for (int i = 0; !*failed; ++i) {
            Patience patience(limit);
            while (*published <= i && !patience.spent(failed))
                __nanosleep(32);
            if (*failed)
                break;
            __threadfence_block();
            const int64_t r = sh.queue[i % ROW_Q].r;
            if (sh.queue[i % ROW_Q].state == ROW_END)
                break;
            const T *row = static_cast<const T *>(a.x) + r * a.ld;
            const int h = head_elems<DT>(row, a.len), nvec = (a.len - h) / E;
            const int nb = batches(nvec), total = nb + twice(nb);
            row += h;
            for (int k = 0; k < total; ++k) {
                const int v0 = (k < nb ? k : k - nb) * U * NT;
                const int n = nvec - v0 < U * NT ? nvec - v0 : U * NT;
                // (after a failure a slot may be given back with its copy in flight)
                if (!mbar_wait(&sh.empty[slot], parity, failed, limit) || *failed)
                    break;
                mbar_expect(&sh.full[slot], (uint32_t)n * 16u);
                bulk_load(ring + slot * U * NT, row + (int64_t)v0 * E, (uint32_t)n * 16u, &sh.full[slot]);
                if (++slot == slots) {
                    slot = 0;
                    parity ^= 1;
                }
            }
        }
        // after a failure the consumers no longer wait for the copies in flight
        if (*failed)
            for (int k = 0; k < slots; ++k)
                for (int n = 0; n < 65536 && !mbar_try(&sh.full[k], k < slot ? parity ^ 1 : parity); ++n)
                    __nanosleep(64);
    } else if (OP::STATS && !OP::TEACHER && warp == NW + 2) {
        // ---- writer
        first_barrier();
        for (int i = 0;; ++i) {
            RowEntry e = sh.queue[i % ROW_Q];
            if (e.state == ROW_END)
                break;
            op.template touch<DT>(a, e);
            const RowStat t = give_row(i, e, 0.0f);
            if (lane == 0)
                op.template write<DT>(a, e, t);
        }
    } else if (OP::TEACHER && warp > NW + 1) {
        if constexpr (OP::TEACHER) {
            // ---- teacher warp w: rows w, w + TEACHERS, ...
            const int w = warp - NW - 2;
            TeacherRow list(lists + (size_t)w * 16 * teacher_k, teacher_k);
            first_barrier();
            for (int i = 0;; ++i) {
                // entries are there a few rows ahead; walk to this warp's next
                const RowEntry e = sh.queue[i % ROW_Q];
                if (e.state == ROW_END)
                    break;
                if (i % TEACHERS != w)
                    continue;
                op.template prepare<DT, 32>(a, e.r, true, list);
                const RowStat t = give_row(i, e, list.mass);
                op.template finish<32>(a, e, t, list);
                if (a.dx) {
                    const RowGrad g = op.template grad<DT>(a, e, t, list.mass);
                    bar_sync(done(i), NT + 32);
                    if (!g.zero)
                        op.template patch<DT, 32>(a, e, g, list, 0, a.len);
                }
                __syncwarp();
            }
        }
    } else if (warp < NW) {
        // ---- consumers
        const T *const x = static_cast<const T *>(a.x);
        T *const dx = static_cast<T *>(a.dx);
        int cslot = 0;  // slot of the next batch, and the phase it arrives in
        uint32_t cphase = 0;
        auto await_batch = [&]() { mbar_wait(&sh.full[cslot], cphase, failed, limit); };
        auto step_slot = [&]() {
            if (++cslot == slots) {
                cslot = 0;
                cphase ^= 1;
            }
        };
        auto release = [&](int slot) {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.empty[slot]);
        };

        first_barrier();
        for (int i = 0;; ++i) {
            if (sh.queue[i % ROW_Q].state == ROW_END)
                break;
            const int64_t r = sh.queue[i % ROW_Q].r;
            const T *const row = x + r * a.ld;
            const int h = head_elems<DT>(row, a.len);
            const int nvec = (a.len - h) / E, nb = batches(nvec), n1 = twice(nb);
            // the row's ragged ends: threads 0..7 the head, 8..15 the tail
            int edge = -1;
            if (tid < h)
                edge = tid;
            else if (tid >= 8 && tid < 16 && h + nvec * E + tid - 8 < a.len)
                edge = h + nvec * E + tid - 8;
            float xe = 0.0f;
            if (edge >= 0)
                xe = load_elem<DT>(row, edge);

            // whether all of the warp's vectors of batch b are within the row
            auto whole = [&](int b) { return nvec - b * U * NT - (tid | 31) > (U - 1) * NT; };

            const int first = cslot;
            if constexpr (OP::STATS) {
                SoftRun run;
                run.init(NEG_INF, s2);
                for (int b = 0; b < nb; ++b) {
                    const uint4 *src = ring + cslot * U * NT + tid;
                    const int left = nvec - b * U * NT - tid;
                    await_batch();
                    uint4 v[U];
                    if (whole(b)) {
                        float top = NEG_INF;
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            v[u] = src[u * NT];
                            top = fmaxf(top, vec_max<DT>(v[u]));
                        }
                        run.raise(top, s2);
                        run.template add<DT, U>(v, s2);
                    } else {
#pragma unroll 1
                        for (int u = 0; u < U && u * NT < left; ++u) {
                            const uint4 w[1] = {src[u * NT]};
                            run.raise(vec_max<DT>(w[0]), s2);
                            run.template add<DT, 1>(w, s2);
                        }
                    }
                    if (!dx || b < n1)
                        release(cslot);
                    step_slot();
                }
                if (edge >= 0) {
                    run.raise(xe, s2);
                    run.add(xe, s2);
                }
                const SoftStat w = soft_warp(run.stat(), s2);
                if (lane == 0)
                    sh.part[i % 2][warp] = w;
            }
            RowGrad g;
            if constexpr (OP::STATS)
                bar_arrive(summed(i), NT + 32);
            else
                g = op.template grad<DT>(a, sh.queue[i % ROW_Q], RowStat{}, 0.0f);
            bar_sync(given(i), GIVEN);
            if (!dx)
                continue;
            if constexpr (OP::STATS)
                g = sh.grad;
            T *const grow = dx + r * a.ldd;
            const bool aligned = ((uintptr_t)(grow + h) & 15u) == 0;
            auto emit = [&](int b, int slot) {
                const uint4 *src = ring + slot * U * NT + tid;
                const int c0 = h + (b * U * NT + tid) * E;
                const int left = nvec - b * U * NT - tid;
                uint4 v[U];
                if (g.zero) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (u * NT < left)
                            store_vec<DT>(grow + c0 + u * NT * E, make_uint4(0, 0, 0, 0), aligned);
                    release(slot);
                } else if (aligned && !g.far && whole(b)) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        v[u] = src[u * NT];
                    release(slot);
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        *reinterpret_cast<uint4 *>(grow + c0 + u * NT * E) = vec_grad<DT>(v[u], g, c0 + u * NT * E);
                } else {
#pragma unroll 1
                    for (int u = 0; u < U && u * NT < left; ++u)
                        store_vec<DT>(grow + c0 + u * NT * E, vec_grad<DT, true>(src[u * NT], g, c0 + u * NT * E), aligned);
                    release(slot);
                }
            };
            if constexpr (OP::STATS) {
                int slot = (first + n1) % slots;
                for (int b = n1; b < nb; ++b) {
                    emit(b, slot);
                    slot = slot + 1 == slots ? 0 : slot + 1;
                }
            }
            // what is fetched for the gradient alone
            for (int b = 0; b < (OP::STATS ? n1 : nb); ++b) {
                await_batch();
                emit(b, cslot);
                step_slot();
            }
            // Not looked at per batch: with the coefficients changed there, policy
            // 1000 x 32001 f32 took 48.3 us instead of 45.0.
            if ((!OP::STATS || n1 > 0) && *failed)
                for (int b = 0; b < (OP::STATS ? n1 : nb); ++b)
                    for (int v = b * U * NT + tid; v < nvec && v < (b + 1) * U * NT; v += NT)
                        store_vec<DT>(grow + h + v * E, nan_vec(), false);
            if (edge >= 0)
                store_elem<DT>(grow, edge, g.zero ? 0.0f : elem_grad<DT>(xe, g, edge));
            if constexpr (OP::TEACHER) {
                bar_arrive(done(i), NT + 32);
            }
        }
    }
}

// ------------------------------------------------------------------ totals

// The CTA's N sums by way of s[N * NT / 32], rounded to out[0, N).
template <int N, int NT>
__device__ void cta_totals(Sum (&v)[N], Sum *s, float *out)
{
    constexpr int NW = NT / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i].join_warp();
        if (lane == 0)
            s[i * NW + warp] = v[i];
    }
    __syncthreads();
    if (threadIdx.x < N) {
        Sum t;
        for (int w = 0; w < NW; ++w)
            t.add(s[threadIdx.x * NW + w]);
        out[threadIdx.x] = t.value();
    }
}

// What remains of a loss when all rows are done, by one CTA of NT threads; s
// has room for 4 sums per warp.
template <class OP, int NT>
__device__ void run_tail(int64_t rows, int len, const OP &op, Sum *s)
{
    if constexpr (OP::TOTALS > 0) {
        Sum v[OP::TOTALS];
        for (int64_t r = threadIdx.x; r < rows; r += NT)
            op.total(r, len, v);
        cta_totals<OP::TOTALS, NT>(v, s, op.stats);
    } else {
        op.template tail<NT>(rows, len, s);
    }
}

constexpr int TOTAL_NT = 256, TOTAL_CTAS = 256, TOTAL_ROWS = 256;

// Totals over rows from the results that a row kernel left: each CTA sums its
// rows, the CTA that finishes last the CTAs' parts, in a fixed order.
template <class OP>
__global__ void __launch_bounds__(TOTAL_NT) total_kernel(int64_t rows, int len, OP op, Sum *part, unsigned *tick)
{
    constexpr int N = OP::TOTALS;
    __shared__ Sum s[N][TOTAL_NT / 32];
    __shared__ bool s_last;
    const int tid = threadIdx.x;
    pdl_enter();
    Sum v[N];
    for (int64_t r = (int64_t)blockIdx.x * TOTAL_NT + tid; r < rows; r += (int64_t)gridDim.x * TOTAL_NT)
        op.total(r, len, v);
    if (gridDim.x == 1) {
        cta_totals<N, TOTAL_NT>(v, s[0], op.stats);
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i].join_warp();
        if ((tid & 31) == 0)
            s[i][tid >> 5] = v[i];
    }
    __syncthreads();
    if (tid < N) {
        Sum t;
        for (int w = 0; w < TOTAL_NT / 32; ++w)
            t.add(s[tid][w]);
        part[(int64_t)blockIdx.x * N + tid] = t;
        __threadfence();
    }
    __syncthreads();
    if (tid == 0)
        s_last = atomicAdd(tick, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!s_last)
        return;
    __threadfence();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = Sum{};
        if (tid < gridDim.x)
            v[i] = part[(int64_t)tid * N + i];
    }
    __syncthreads();  // (s is free again)
    cta_totals<N, TOTAL_NT>(v, s[0], op.stats);
    if (tid == 0)
        *tick = 0;
}

// ------------------------------------------------------------- short rows

constexpr int GROUP_NT = 256;

// G lanes per row, the row in registers (NV vectors per lane): rows too short
// for a CTA barrier each.  The shorter the row, the fewer the lanes, so that
// what is done once per row (the loss itself, its logarithms and exponentials,
// the reductions) is done for 32 / G rows at a time; two warps (G = 64) join
// their statistics by way of shared memory and a barrier of their own.  The next row's entry is
// fetched while this row is at work, and so is (STAGED) the next row.
template <int DT, class OP, int G, int NV, bool STAGED>
__global__ void __launch_bounds__(GROUP_NT, NV > 8 ? 2 : 3) group_row_kernel(LogitRows a, OP op, int teacher_k)
{
    using T = typename Elem<DT>::T;
    constexpr int E = VEC_ELEMS<DT>;
    constexpr int ROWS = GROUP_NT / G;  // rows of a CTA at a time
    extern __shared__ __align__(16) unsigned char smem[];
    const int gl = threadIdx.x & (G - 1), group = threadIdx.x / G;
    uint4 *const stage = reinterpret_cast<uint4 *>(smem) + threadIdx.x;  // of this lane, GROUP_NT apart
    TeacherRow list(smem + (STAGED ? NV * GROUP_NT * 16 : 0) + (size_t)group * 16 * teacher_k, teacher_k);
    const float s2 = a.s2;
    const T *const x = static_cast<const T *>(a.x);
    T *const dx = static_cast<T *>(a.dx);
    pdl_enter();

    const int64_t step = (int64_t)gridDim.x * ROWS;
    // The entry of the next row, and (if STAGED) that row on its way into shared
    // memory: each lane fetches and reads its own vectors, so no other waits.
    RowEntry n{};
    constexpr int ENDS = (2 * (E - 1) + G - 1) / G;  // the row's ragged ends, fewer than E elements each
    float n_x[ENDS];
    auto end_at = [&](int k, int h, int nvec) {
        const int i = gl + k * G, tail = a.len - h - nvec * E;
        return i < h ? i : (i - h < tail ? a.len - tail + i - h : -1);
    };
    auto load = [&](int64_t r, RowEntry &to) {
        to.state = ROW_END;
        if (r < a.rows) {
            op.load(r, to);
            to.state = ROW_LIVE;
        }
    };
    auto settle = [&]() {
        if (n.state != ROW_END) {
            op.settle(a, n);
            if (n.state == ROW_LIVE)
                op.template touch<DT>(a, n);
        }
    };
    auto load_ends = [&](const T *row, int h, int nvec) {
#pragma unroll
        for (int k = 0; k < ENDS; ++k) {
            const int j = end_at(k, h, nvec);
            n_x[k] = j >= 0 ? load_elem<DT>(row, j) : NEG_INF;
        }
    };
    auto request = [&]() {
        if (STAGED && n.state == ROW_LIVE) {
            const T *const row = x + n.r * a.ld;
            const int h = head_elems<DT>(row, a.len), nvec = (a.len - h) / E;
            const uint4 *const vec = reinterpret_cast<const uint4 *>(row + h) + gl;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i * G + gl < nvec)
                    async_load16(stage + i * GROUP_NT, vec + i * G);
            load_ends(row, h, nvec);
        }
    };
    // The maximum and the sum of two warps' values: each is read between its own
    // barrier and the other's next, and written after that.
    __shared__ float s_max[GROUP_NT / 32], s_sum[GROUP_NT / 32];
    const int warp = threadIdx.x / 32;
    auto join_max = [&](float v) {
        s_max[warp] = v;
        bar_sync(1 + group, G);
#pragma unroll
        for (int k = 0; k < G / 32; ++k)
            v = fmaxf(v, s_max[group * (G / 32) + k]);
        return v;
    };
    auto join_sum = [&](float v) {
        s_sum[warp] = v;
        bar_sync(1 + group, G);
        v = 0.0f;
#pragma unroll
        for (int k = 0; k < G / 32; ++k)
            v += s_sum[group * (G / 32) + k];
        return v;
    };
    // (the loop is the same for all of a warp: its first group has the first row)
    constexpr int PER_WARP = G < 32 ? 32 / G : 1;
    int64_t r0 = (int64_t)blockIdx.x * ROWS + (group & ~(PER_WARP - 1));
    const int sub = group & (PER_WARP - 1);
    load(r0 + sub, n);
    settle();
    request();
    for (; r0 < a.rows; r0 += step) {
        const RowEntry e = n;
        const bool live = e.state == ROW_LIVE;
        const T *const row = x + e.r * a.ld;
        const int h = head_elems<DT>(row, a.len), nvec = (a.len - h) / E;
        uint4 v[NV];
        float end_x[ENDS];
        if (!STAGED && live)
            load_ends(row, h, nvec);
#pragma unroll
        for (int k = 0; k < ENDS; ++k)
            end_x[k] = n_x[k];
        load(r0 + sub + step, n);
        if (STAGED)
            async_wait();
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i * G + gl < nvec)
                    v[i] = STAGED ? stage[i * GROUP_NT] : reinterpret_cast<const uint4 *>(row + h)[i * G + gl];
        }
        settle();
        request();
        if constexpr (OP::TEACHER)
            op.template prepare<DT, G>(a, e.r, live, list);

        RowStat t{};
        if constexpr (OP::STATS) {
            float top = NEG_INF;
            if (live) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (i * G + gl < nvec)
                        top = fmaxf(top, vec_max<DT>(v[i]));
#pragma unroll
                for (int k = 0; k < ENDS; ++k)
                    top = fmaxf(top, end_x[k]);
            }
            top = G > 32 ? join_max(group_max<32>(top)) : group_max<G>(top);
            SoftRun run;
            run.init(top, s2);
            if (live && is_near(run.m2)) {
                const f32x2 sa = pack2(s2, s2), sb = pack2(-run.m2, -run.m2);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (i * G + gl < nvec)
                        run.template add_near<DT>(v[i], sa, sb);
            } else if (live) {
                for (int i = gl; i < nvec; i += G)
                    run.l = SoftRun::template far_sum<DT>(reinterpret_cast<const uint4 *>(row + h)[i], top, s2, run.l);
            }
            if (live) {
#pragma unroll
                for (int k = 0; k < ENDS; ++k)
                    run.add(end_x[k], s2);
            }
            const float l = run.stat().l;
            t = row_stat(a, SoftStat{top, G > 32 ? join_sum(group_sum<32>(l)) : group_sum<G>(l)});
        }
        if constexpr (OP::TEACHER)
            op.template finish<G>(a, e, t, list);
        else if (gl == 0 && live)
            op.template write<DT>(a, e, t);
        if (gl == 0 && e.state == ROW_OUT)
            op.skip(e.r);
        if (!dx)
            continue;
        T *const grow = dx + e.r * a.ldd;
        RowGrad g = op.template grad<DT>(a, e, t, list.mass);
        g.zero = g.zero || !live;
        const bool aligned = ((uintptr_t)(grow + h) & 15u) == 0;
        if (!g.zero && !g.far && aligned) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i * G + gl < nvec) {
                    const int j = h + (i * G + gl) * E;
                    *reinterpret_cast<uint4 *>(grow + j) = vec_grad<DT>(v[i], g, j);
                }
        } else if (e.state != ROW_END) {
            // rarer rows, one vector at a time from memory again
            for (int i = gl; i < nvec; i += G) {
                const int j = h + i * E;
                store_vec<DT>(grow + j, g.zero ? make_uint4(0, 0, 0, 0)
                                               : vec_grad<DT, true>(*reinterpret_cast<const uint4 *>(row + j), g, j),
                              aligned);
            }
        }
        if (e.state != ROW_END) {
#pragma unroll
            for (int k = 0; k < ENDS; ++k) {
                const int j = end_at(k, h, nvec);
                if (j >= 0)
                    store_elem<DT>(grow, j, g.zero ? 0.0f : elem_grad<DT>(end_x[k], g, j));
            }
        }
        if constexpr (OP::TEACHER) {
            __syncwarp();
            if (!g.zero)
                op.template patch<DT, G>(a, e, g, list, 0, a.len);
            __syncwarp();
        }
    }
}

// --------------------------------------------------------------- few rows

constexpr int FEW_NT = 256, FEW_NW = FEW_NT / 32, MAX_CLUSTER = 8;

// A cluster of CTAs per row, a slice of the columns each, held in registers
// (NV vectors per thread): few rows, for which latency counts.  All loads are
// out at once, the statistics of the slices meet through distributed shared
// memory, and the CTA that finishes last sums the totals.
template <int DT, class OP, int NV>
__global__ void __launch_bounds__(FEW_NT) few_row_kernel(LogitRows a, OP op, int teacher_k, unsigned *tick)
{
    using T = typename Elem<DT>::T;
    constexpr int E = VEC_ELEMS<DT>;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ SoftStat s_part[FEW_NW], s_slice[MAX_CLUSTER];
    __shared__ float s_mass;
    __shared__ bool s_last;
    TeacherRow list(smem, teacher_k);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cs = cluster_size(), rank = cluster_rank();
    const float s2 = a.s2;
    cluster_arrive();
    pdl_enter();

    RowEntry e;
    op.load(blockIdx.x / cs, e);
    const int64_t r = e.r;
    const T *const row = static_cast<const T *>(a.x) + r * a.ld;
    T *const grow = static_cast<T *>(a.dx) + r * a.ldd;
    const int h = head_elems<DT>(row, a.len), all = (a.len - h) / E;
    const int q = (all + cs - 1) / cs, begin = min(rank * q, all), n = min(q, all - begin);
    const int j0 = h + begin * E;  // first column of the slice
    uint4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i * FEW_NT + tid < n)
            v[i] = reinterpret_cast<const uint4 *>(row + j0)[i * FEW_NT + tid];
    // the row's ragged ends: the first CTA's threads 0..7, the last one's 8..15
    int edge = -1;
    if (rank == 0 && tid < h)
        edge = tid;
    else if (rank == cs - 1 && tid >= 8 && tid < 16 && h + all * E + tid - 8 < a.len)
        edge = h + all * E + tid - 8;
    float xe = 0.0f;
    if (edge >= 0)
        xe = load_elem<DT>(row, edge);
    op.settle(a, e);
    if (e.state == ROW_LIVE)
        op.template touch<DT>(a, e);

    RowStat t{};
    if (e.state == ROW_LIVE) {
        if constexpr (OP::TEACHER) {
            if (warp == 0) {
                op.template prepare<DT, 32>(a, r, true, list);
                if (lane == 0)
                    s_mass = list.mass;
            }
        }
        if constexpr (OP::STATS) {
            SoftRun run;
            float top = edge >= 0 ? fmaxf(xe, NEG_INF) : NEG_INF;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i * FEW_NT + tid < n)
                    top = fmaxf(top, vec_max<DT>(v[i]));
            run.init(top, s2);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i * FEW_NT + tid < n) {
                    const uint4 w[1] = {v[i]};
                    run.template add<DT, 1>(w, s2);
                }
            if (edge >= 0)
                run.add(xe, s2);
            SoftStat w = soft_warp(run.stat(), s2);
            if (lane == 0)
                s_part[warp] = w;
            __syncthreads();
            w = soft_warp<FEW_NW>(s_part[lane % FEW_NW], s2);
            cluster_wait();  // for the others to have started
            if (tid < cs)
                *in_cta(&s_slice[rank], tid) = w;
            cluster_arrive();
            cluster_wait();
            w = soft_warp<MAX_CLUSTER>(s_slice[lane % cs], s2);
            w.l *= (float)cs / MAX_CLUSTER;  // (every slice was there MAX_CLUSTER / cs times)
            t = row_stat(a, w);
        }
    }
    if (rank == 0 && warp == 0) {
        if (e.state == ROW_OUT) {
            if (tid == 0)
                op.skip(r);
        } else if constexpr (OP::TEACHER) {
            op.template finish<32>(a, e, t, list);
        } else if (tid == 0) {
            op.template write<DT>(a, e, t);
        }
        if (OP::TAIL && tid == 0) {
            __threadfence();
            s_last = atomicAdd(tick, 1u) == (unsigned)a.rows - 1;
        }
    }
    if (a.dx && e.state == ROW_LIVE) {
        const RowGrad g = op.template grad<DT>(a, e, t, OP::TEACHER ? s_mass : 0.0f);
        const bool aligned = ((uintptr_t)(grow + h) & 15u) == 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i * FEW_NT + tid < n) {
                const int j = j0 + (i * FEW_NT + tid) * E;
                const uint4 o = g.zero ? make_uint4(0, 0, 0, 0)
                                       : (g.far ? vec_grad<DT, true>(v[i], g, j) : vec_grad<DT>(v[i], g, j));
                store_vec<DT>(grow + j, o, aligned);
            }
        if (edge >= 0)
            store_elem<DT>(grow, edge, g.zero ? 0.0f : elem_grad<DT>(xe, g, edge));
        if constexpr (OP::TEACHER) {
            __syncthreads();
            if (warp == 0 && !g.zero)
                op.template patch<DT, 32>(a, e, g, list, rank == 0 ? 0 : j0, rank == cs - 1 ? a.len : j0 + n * E);
        }
    } else if (a.dx) {
        zero_row<DT>(grow, a.len, rank * FEW_NT + tid, cs * FEW_NT);
    }
    if constexpr (OP::TAIL) {
        __shared__ Sum s_sum[4 * FEW_NW];
        if (rank != 0)
            return;
        __syncthreads();
        if (!s_last)
            return;
        __threadfence();
        run_tail<OP, FEW_NT>(a.rows, a.len, op, s_sum);
        if (tid == 0)
            *tick = 0;
    }
}

// --------------------------------------------------------------- launchers

// Launch with dynamic shared memory, programmatic serialization (as
// launch_pdl) and clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_smem(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                            cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Longest row of the group kernel.
constexpr size_t GROUP_ROW_BYTES = 8192;
// Longest row of two warps of it.
constexpr size_t PAIR_ROW_BYTES = 16384;

// The few-row kernel is taken while its CTAs, with the largest cluster that
// allows it, are at most this many per two SMs (and a thread's slice 8
// vectors).  us, few-row kernel against the row kernel: logprob 1 x 65536 bf16
// 2.4 / 5.9, 64 rows 4.6 / 6.3; policy 1 row 5.5 / 9.4, 30 rows 6.3 / 9.5, 64
// rows 8.0 / 9.4, 100 rows 9.4 / 9.8, 300 x 16384 f32 9.4 / 10.5.  With 4
// CTAs per SM they no longer all run at once: 152 x 65536 bf16 12.5 / 10.1.
// Against two warps of the group kernel: logprob 20 x 8100 bf16 2.8 / 3.8, 250 x
// 8100 4.4 / 4.5, 250 x 4200 4.1 / 3.1; preference 250 x 4200 11.8 / 12.4.
constexpr int FEW_CTAS_PER_2_SMS = 7;

constexpr size_t SM_SMEM = 228 * 1024, CTA_SMEM = 227 * 1024, CTA_RESERVED = 1024;
constexpr size_t FEW_SMEM = CTA_SMEM - 1024;  // beside the few-row kernel's static part

template <int DT, class OP, int NT, int U>
int launch_row_kernel(const LogitRows &a, const OP &op, int per_sm, int teacher_k, cudaStream_t s, const DeviceInfo &di)
{
    Workspace ws;
    const int st = get_workspace(&ws);
    if (st != RED_OK)
        return st;
    constexpr int SERVICE = 32 * SERVICE_WARPS<OP>;
    constexpr size_t batch = (size_t)U * NT * 16;
    const size_t fixed = sizeof(RowShared<NT / 32>) + (size_t)TEACHERS * 4 * 4 * teacher_k;
    size_t most = SM_SMEM / per_sm - CTA_RESERVED;
    most = most < CTA_SMEM ? most : CTA_SMEM;
    int slots = most > fixed ? (int)((most - fixed) / batch) : 0;
    slots = slots < ROW_MAX_SLOTS ? slots : ROW_MAX_SLOTS;
    if (slots < 2)
        slots = 2;
    const size_t smem = slots * batch + fixed;
    const auto kernel = row_kernel<DT, OP, NT, U>;
    static std::atomic<uint64_t> ready{0};  // a bit per device
    if (!(ready.load(std::memory_order_relaxed) >> di.dev & 1)) {
        const cudaError_t e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)CTA_SMEM);
        if (e != cudaSuccess)
            return cuda_fail(e, "row kernel: shared memory");
        ready.fetch_or(uint64_t(1) << di.dev, std::memory_order_relaxed);
    }
    const int64_t cap = (int64_t)di.sms * per_sm;
    const unsigned grid = (unsigned)(a.rows < cap ? a.rows : cap);
    // Rows taken at a time: one, except short ones, which the counter's latency
    // would hold up where many are out of the loss (policy 20000 x 8192 bf16, 40%
    // of them: 91 us with two, 96 with one; 8192 x 65536: 283 and 278).
    const int group = a.len * (int64_t)sizeof(typename Elem<DT>::T) <= 24576 ? 2 : 1;
    const int ahead = OP::TEACHER ? TEACHERS : 0;
    const cudaError_t e = launch_pdl_smem(kernel, grid, NT + SERVICE, smem, 1, s, a, op, ws.tick, slots,
                                          group, ahead, teacher_k, (unsigned)knob(RED_KNOB_LOSS_TRIES));
    count_launches(1);
    return cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "row kernel launch");
}

template <int DT, class OP, int G, int NV, bool STAGED>
int launch_group_kernel(const LogitRows &a, const OP &op, int teacher_k, cudaStream_t s, const DeviceInfo &di)
{
    const auto kernel = group_row_kernel<DT, OP, G, NV, STAGED>;
    constexpr int ROWS = GROUP_NT / G;
    constexpr int STAGE = STAGED ? NV * GROUP_NT * 16 : 0;
    const size_t smem = STAGE + (size_t)ROWS * 16 * teacher_k;
    // residency, kept per instance for the last device and list length asked for
    static std::atomic<int64_t> known{-1};
    const int64_t want_key = (int64_t)di.dev << 24 | teacher_k;
    int64_t k = known.load(std::memory_order_relaxed);
    if (k < 0 || (k >> 8) != want_key) {
        cudaError_t e = cudaSuccess;
        if (smem > 47 * 1024)  // 48 KB with the static part
            e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     STAGE + GROUP_NT / 32 * 16 * RED_DISTILL_MAX_K);
        int occ = 0;
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, (const void *)kernel, GROUP_NT, smem);
        if (e != cudaSuccess || occ < 1)
            return e != cudaSuccess ? cuda_fail(e, "row group kernel: occupancy")
                                    : fail(RED_ECUDA, "row group kernel cannot be resident on this device");
        k = want_key << 8 | occ;
        known.store(k, std::memory_order_relaxed);
    }
    const int64_t want = (a.rows + ROWS - 1) / ROWS, cap = di.sms * (k & 255);
    const cudaError_t e =
        launch_pdl_smem(kernel, (unsigned)(want < cap ? want : cap), GROUP_NT, smem, 1, s, a, op, teacher_k);
    count_launches(1);
    return cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "row group kernel launch");
}

template <int DT, class OP, int NV>
int launch_few_kernel(const LogitRows &a, const OP &op, int cluster, int teacher_k, cudaStream_t s,
                      const DeviceInfo &di)
{
    Workspace ws;
    const int st = get_workspace(&ws);
    if (st != RED_OK)
        return st;
    const auto kernel = few_row_kernel<DT, OP, NV>;
    static std::atomic<uint64_t> ready{0};  // a bit per device
    if (!(ready.load(std::memory_order_relaxed) >> di.dev & 1)) {
        const cudaError_t e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)FEW_SMEM);
        if (e != cudaSuccess)
            return cuda_fail(e, "few-row kernel: shared memory");
        ready.fetch_or(uint64_t(1) << di.dev, std::memory_order_relaxed);
    }
    // Shared memory that leaves room on an SM for its share of the CTAs and no
    // more: left to themselves clusters crowd some SMs and leave others idle.  us
    // without and with: policy 64 x 65536 bf16 8.8, 7.9; 30 x 65536 7.4, 6.3; 200 x
    // 32001 9.8, 8.8; logprob_grad 200 x 32000 4.3, 3.8; 120 x 50257 unchanged.
    const int64_t ctas = a.rows * cluster, share = (ctas + di.sms - 1) / di.sms;
    const size_t list = (size_t)4 * 4 * teacher_k, part = SM_SMEM / share - 2 * CTA_RESERVED;
    const size_t smem = list > part ? list : (part < FEW_SMEM ? part : FEW_SMEM);
    const cudaError_t e = launch_pdl_smem(kernel, (unsigned)ctas, FEW_NT, smem, (unsigned)cluster, s, a, op,
                                          teacher_k, ws.tick);
    count_launches(1);
    return cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "few-row kernel launch");
}

template <class OP>
int launch_totals(const LogitRows &a, const OP &op, cudaStream_t s)
{
    if constexpr (OP::TOTALS > 0) {
        Workspace ws;
        const int st = get_workspace(&ws);
        if (st != RED_OK)
            return st;
        const int64_t want = (a.rows + TOTAL_ROWS - 1) / TOTAL_ROWS;
        const cudaError_t e = launch_pdl(total_kernel<OP>, dim3((unsigned)(want < TOTAL_CTAS ? want : TOTAL_CTAS)),
                                         dim3(TOTAL_NT), s, a.rows, a.len, op, static_cast<Sum *>(ws.part), ws.tick);
        count_launches(1);
        return cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "totals launch");
    }
    return RED_OK;
}

// Rows longer than the group kernel's, where they are few: *taken, and what
// remains after the rows is done, too.
template <int DT, class OP>
int launch_few(const LogitRows &a, const OP &op, int teacher_k, cudaStream_t s, const DeviceInfo &di, bool *taken)
{
    const size_t bytes = (size_t)a.len * sizeof(typename Elem<DT>::T);
    const int64_t nvec = (int64_t)(bytes / 16);
    for (int cluster = MAX_CLUSTER; bytes > GROUP_ROW_BYTES && cluster >= 2; cluster /= 2) {
        const int64_t slice = (nvec + cluster - 1) / cluster;
        if (2 * a.rows * cluster > FEW_CTAS_PER_2_SMS * di.sms || slice > 8 * FEW_NT)
            continue;
        *taken = true;
        return slice <= 4 * FEW_NT ? launch_few_kernel<DT, OP, 4>(a, op, cluster, teacher_k, s, di)
                                   : launch_few_kernel<DT, OP, 8>(a, op, cluster, teacher_k, s, di);
    }
    return RED_OK;
}

// Many rows per group of lanes have the next one fetched into shared memory
// while one is at work.  us without and with, at 1.3, 2.6, 3.8 and 6 rows per
// group: policy of 1000 bf16 logits 13.6 13.3, 23.1 22.2, 32.4 29.5, 43.5 39.7;
// of 8000 16.5 16.4, 29.4 25.5, 38.5 33.6, 53.1 45.9; logprob of 350 5.3 5.8,
// 8.1 8.8, 11.9 11.3, 20.2 17.9.  Not for the gradient alone, which has little
// else to do (14592 x 4000 39.8 38.0, 43776 x 1000 29.4 29.5), not where the
// lists of a teacher want the space and the row in L1 (distill 30000 x 400, 64
// entries: 50.5 64.5), nor for the shortest rows, for want of registers (policy
// 65536 x 120 16.1 17.7).
template <int DT, class OP, int G, int NV>
int launch_group(const LogitRows &a, const OP &op, int teacher_k, cudaStream_t s, const DeviceInfo &di)
{
    if constexpr (OP::STATS && !OP::TEACHER && G > 4) {
        const int64_t resident = (int64_t)di.sms * (NV > 8 ? 2 : 3) * (GROUP_NT / G);
        if (a.rows > 3 * resident)
            return launch_group_kernel<DT, OP, G, NV, true>(a, op, teacher_k, s, di);
    }
    return launch_group_kernel<DT, OP, G, NV, false>(a, op, teacher_k, s, di);
}

// All rows, by the kernel for their number and length; *finished: what remains
// after them is done, too.
template <int DT, class OP>
int launch_rows_of(const LogitRows &a, const OP &op, int teacher_k, cudaStream_t s, bool *finished)
{
    DeviceInfo di;
    int st = device_info(&di);
    if (st == RED_OK)
        st = launch_few<DT>(a, op, teacher_k, s, di, finished);
    if (st != RED_OK || *finished)
        return st;
    const size_t bytes = (size_t)a.len * sizeof(typename Elem<DT>::T);
    auto fits = [&](int lanes, int vectors) { return bytes <= (size_t)lanes * vectors * 16; };
    if (bytes <= GROUP_ROW_BYTES) {
        // Lanes per row.  Many rows: as few as hold the row, up to 8 vectors each
        // (what is done once per row is then done for more of them at a time), but
        // enough for the teacher's list.  Few rows: as many as let all rows run at
        // once.  us with 4, 8, 16 and 32 lanes (- where 4 do not hold the row):
        //   policy       500 x 250 bf16      8.4    7.4    6.9    7.0
        //               3600 x 250           9.2    9.0    8.1    9.2
        //               7000 x 250          10.7    9.4    8.8   11.3
        //              15000 x 250          11.7   11.4   13.2   17.8
        //              30000 x 120          11.5   12.7   17.1   28.7
        //               7000 x 500             -   10.9    9.4   11.8
        //              30000 x 500             -   18.9   22.4   33.0
        //   distill 30000 x 120, k = 4      13.1   15.9   22.8   37.1
        //                        k = 16     22.6   19.9   24.3   40.6
        //                        k = 64     68.2   38.5   34.9   49.3
        //   logprob_grad 3600 x 500            -    3.7    2.9    2.8
        int lanes = fits(4, 8) ? 4 : fits(8, 8) ? 8 : fits(16, 8) ? 16 : 32;
        while (lanes < 16 && teacher_k > lanes * lanes / 2)
            lanes *= 2;
        while (lanes < 32 && a.rows <= (int64_t)di.sms * 3 * (GROUP_NT / (2 * lanes)))
            lanes *= 2;
        // room for the lists of a second CTA's rows
        while (lanes < 32 && (size_t)(GROUP_NT / lanes) * 16 * teacher_k > 96 * 1024)
            lanes *= 2;
        if (lanes == 4)
            return launch_group<DT, OP, 4, 8>(a, op, teacher_k, s, di);
        if (lanes == 8)
            return launch_group<DT, OP, 8, 8>(a, op, teacher_k, s, di);
        if (lanes == 16)
            return launch_group<DT, OP, 16, 8>(a, op, teacher_k, s, di);
        // Registers for 12 vectors where the row needs no more, us against the next
        // form: policy 22882 x 576 f32 25.7, 30.5; 60000 x 1300 bf16 77.8, 82.2;
        // 60000 x 2400 116, 123; logprob 60000 x 2400 55.2, 62.0.  Half a warp only
        // for many rows (policy 2500 x 1056 bf16 8.9, 8.6), and not for a teacher's
        // lists and the gradient alone (distill 60000 x 1300 142, 138; logprob_grad
        // 54.0, 53.8).
        if constexpr (OP::STATS && !OP::TEACHER)
            if (fits(16, 12) && a.rows > (int64_t)di.sms * 3 * (GROUP_NT / 32))
                return launch_group<DT, OP, 16, 12>(a, op, teacher_k, s, di);
        if (fits(32, 8))
            return launch_group<DT, OP, 32, 8>(a, op, teacher_k, s, di);
        return fits(32, 12) ? launch_group<DT, OP, 32, 12>(a, op, teacher_k, s, di)
                            : launch_group<DT, OP, 32, 16>(a, op, teacher_k, s, di);
    }
    // Two warps per row, us against the row kernel: policy 20000 x 8000 bf16 109,
    // 142; 30000 x 6000 bf16 128, 162; 30000 x 4104 bf16 110, 140; 800 x 5000 bf16
    // 9.6, 11.9; logprob 30000 x 6000 bf16 63, 84.  Four warps for up to 32 KB lose
    // (policy 16000 x 10000 bf16 130, 115), and so do four for up to 16 KB where
    // rows are many (20000 x 4000 f32 112, 106 with two; 800 x 8000 bf16 9.8, 10.7).
    // With 12 vectors per lane and 16: 30000 x 6000 bf16 128, 135.
    if constexpr (OP::STATS && !OP::TEACHER)
        if (bytes <= PAIR_ROW_BYTES)
            return fits(64, 12) ? launch_group<DT, OP, 64, 12>(a, op, teacher_k, s, di)
                                : launch_group<DT, OP, 64, 16>(a, op, teacher_k, s, di);
    // Threads, vectors per thread and batch, and CTAs per SM, by row bytes.  A
    // CTA is busy with one row at a time, so short rows need several CTAs to
    // cover each other's barriers, and long ones a ring that holds a row and
    // the start of the next.  us, policy loss and gradient:
    //                          512x4,1   256x4,2   256x4,3   128x8,4   128x4,4   128x4,6
    //   8192 x 65536 bf16          278       301       332       351       354       368
    //   4096 x 50257 bf16          149       135       150       162       161       161
    //   4096 x 30000 bf16          108        85        83        89        89        91
    //   8192 x 16384 bf16          126        96        86        87        87        93
    //   16384 x 8192 bf16          222       121       103        91        96        97
    // A teacher's list takes time that more rows at once cover: distill 4096 x
    // 16384 bf16 75, 63, 65, 68, 59, 64.  Without a gradient a row need not
    // stay: logprob 4096 x 50257 f16 62, 53, 48, 48, 50, 53; 16384 x 8192 bf16
    // 145, 76, 58, 48, 50, 52.
    // Without statistics nothing does: logprob_grad 3001 x 32001 bf16 54, 54,
    // 55, 56, 56, 54; 32768 x 4100 bf16 250, 133, 104, 92, 86, 87.  (A loss
    // with a gradient keeps its mapping when the gradient is not asked for:
    // the mapping sets the order of the sums.)
    if constexpr (!OP::GRADIENT) {
        return launch_row_kernel<DT, OP, 128, 8>(a, op, 4, teacher_k, s, di);
    } else if constexpr (!OP::STATS) {
        return bytes > 24576 ? launch_row_kernel<DT, OP, 256, 4>(a, op, 2, teacher_k, s, di)
                             : launch_row_kernel<DT, OP, 128, 4>(a, op, 4, teacher_k, s, di);
    } else {
        if (bytes > 122880)
            return launch_row_kernel<DT, OP, 512, 4>(a, op, 1, teacher_k, s, di);
        if (bytes > 40960)
            return launch_row_kernel<DT, OP, 256, 4>(a, op, bytes > 65536 ? 2 : 3, teacher_k, s, di);
        if constexpr (!OP::TEACHER)
            return launch_row_kernel<DT, OP, 128, 8>(a, op, 4, teacher_k, s, di);
        else
            return launch_row_kernel<DT, OP, 128, 4>(a, op, bytes > 12288 ? 4 : 6, teacher_k, s, di);
    }
}

template <class OP>
int launch_loss_rows(int dtype, const LogitRows &a, const OP &op, int teacher_k, cudaStream_t s)
{
    bool finished = false;
    int st;
    switch (dtype) {
    case RED_F32: st = launch_rows_of<RED_F32>(a, op, teacher_k, s, &finished); break;
    case RED_F16: st = launch_rows_of<RED_F16>(a, op, teacher_k, s, &finished); break;
    default: st = launch_rows_of<RED_BF16>(a, op, teacher_k, s, &finished); break;
    }
    return st != RED_OK || finished ? st : launch_totals(a, op, s);
}

}  // namespace red
