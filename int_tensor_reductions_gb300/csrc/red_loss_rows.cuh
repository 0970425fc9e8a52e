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
// A service warp takes rows, reads their scalars (target, weight, the
// target's logit) ahead into a queue, and writes the losses; teacher warps
// do the same for the rows' lists of teacher entries.  One CTA barrier per
// row joins the statistics and hands the queue over.
#pragma once

#include <type_traits>

#include "red_internal.h"
#include "red_loss.cuh"
#include "red_prims.cuh"

namespace red {

// ------------------------------------------------------- vectors of logits

template <int DT>
constexpr int VEC_ELEMS = DT == RED_F32 ? 4 : 8;  // in 16 bytes

__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b)
{
    float2 d;
    asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{ .reg .b64 x, y, z, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7}; "
        "fma.rn.f32x2 w, x, y, z; mov.b64 {%0, %1}, w; }"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// Pair i of a vector, widened.
template <int DT>
__device__ __forceinline__ float2 vec_pair(const uint4 &v, int i)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (DT == RED_F32)
        return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else if constexpr (DT == RED_BF16)
        return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else {
        __half2 h;
        memcpy(&h, &w[i], 4);
        return __half22float2(h);
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
__device__ __forceinline__ uint4 vec_pack(const float2 (&f)[VEC_ELEMS<DT> / 2])
{
    uint4 v;
    if constexpr (DT == RED_F32) {
        v = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                       __float_as_uint(f[1].y));
    } else if constexpr (DT == RED_BF16) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = __float22bfloat162_rn(f[i]);
        memcpy(&v, h, 16);
    } else {
        __half2 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = __float22half2_rn(f[i]);
        memcpy(&v, h, 16);
    }
    return v;
}

// Running statistics of one thread; the sum in two lanes.
struct SoftRun {
    float m;
    float2 l;

    __device__ __forceinline__ void init()
    {
        m = NEG_INF;
        l = make_float2(0.0f, 0.0f);
    }
    __device__ __forceinline__ void raise(float to, float s2)
    {
        to = fmaxf(m, to);
        const float f = ex2((m - ref_of(to)) * s2);
        l = make_float2(l.x * f, l.y * f);
        m = to;
    }
    template <int DT>
    __device__ __forceinline__ void add(const uint4 &v, float s2)
    {
        const float at = ref_of(m);
#pragma unroll
        for (int i = 0; i < VEC_ELEMS<DT> / 2; ++i) {
            const float2 d = mul_f32x2(add_f32x2(vec_pair<DT>(v, i), make_float2(-at, -at)), make_float2(s2, s2));
            l = add_f32x2(l, make_float2(ex2(d.x), ex2(d.y)));
        }
    }
    __device__ __forceinline__ void add(float v, float s2) { l.x += ex2((v - ref_of(m)) * s2); }
    __device__ __forceinline__ SoftStat stat() const { return SoftStat{m, l.x + l.y}; }
};

// The gradient of one vector of logits whose first column is j0.
template <int DT>
__device__ __forceinline__ uint4 vec_grad(const uint4 &v, const RowGrad &g, int j0)
{
    constexpr int E = VEC_ELEMS<DT>;
    float2 o[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        const float2 d = mul_f32x2(fma_f32x2(vec_pair<DT>(v, i), make_float2(g.fa, g.fa), make_float2(g.fb, g.fb)),
                                   make_float2(g.fc, g.fc));
        o[i] = mul_f32x2(make_float2(ex2(d.x), ex2(d.y)), make_float2(g.mul, g.mul));
    }
    const unsigned at = (unsigned)(g.y - j0);
    if (at < (unsigned)E) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            o[i].x += at == 2 * i ? g.cy : 0.0f;
            o[i].y += at == 2 * i + 1 ? g.cy : 0.0f;
        }
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

// No wait is without end: one that runs out (which takes a hardware fault)
// marks the CTA as failed, and its rows' results become NaN.
constexpr int WAIT_TRIES = 1 << 20;

__device__ __forceinline__ void mbar_wait(uint64_t *bar, uint32_t parity, volatile int *failed)
{
    for (int n = 0; !mbar_try(bar, parity); ++n)
        if (n == WAIT_TRIES || ((n & 255) == 255 && *failed)) {
            *failed = 1;
            return;
        }
}

// `bytes` (a multiple of 16) from src to shared memory; both 16-byte aligned.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

constexpr int ROW_Q = 32;      // entries of the row queue
constexpr int ROW_MAX_GROUP = 4;
constexpr int ROW_MAX_SLOTS = 32;
constexpr int TEACHERS = 4;    // teacher warps: each has the time of this many rows for one list

// Shared memory of the row kernel behind the slots.
template <int NW, int PARTS>
struct RowShared {
    RowEntry queue[ROW_Q];
    SoftStat part[PARTS][NW];  // statistics of row i's warps in part[i % PARTS]
    float mass[TEACHERS];  // sum of a row's teacher probabilities
    uint64_t full[ROW_MAX_SLOTS], empty[ROW_MAX_SLOTS];
    int published;  // entries written to the queue
    int loading;    // entry the loader is at
    int failed;     // a wait ran out
};

// A buffer of statistics is written again PARTS rows later: after the next
// barrier of its readers, which for a teacher warp is TEACHERS rows later.
template <class OP>
constexpr int PARTS = OP::TEACHER ? 2 * TEACHERS : 2;

template <class OP>
constexpr int SERVICE_WARPS = OP::TEACHER ? 2 + TEACHERS : 2;  // service, loader, teachers

__device__ __forceinline__ void bar_sync(int id, int n)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// NT consumer threads and the service warps; `slots` batches of U * NT
// vectors in shared memory.  next: the row counter and the count of finished
// CTAs, both zero before and after.
//
// The queue: entry i is in slot i % ROW_Q.  Its first 3 * group + AHEAD
// entries are fixed rows; after that the service warp takes `group` rows at a
// time from the counter, in steps of `group` rows that each advance a chain
// of three loads (counter, scalars, target's logit) by one link, so that no
// step waits for more than one latency: step s, before the barrier of row s *
// group, publishes the group that step s - 3 took.  After the barrier of row
// i at least the entries up to i + AHEAD can be read.
template <int DT, class OP, int NT, int U>
__global__ void __launch_bounds__(NT + 32 * SERVICE_WARPS<OP>)
row_kernel(LogitRows a, OP op, unsigned *next, int slots, int group, int teacher_k)
{
    using T = typename Elem<DT>::T;
    constexpr int E = VEC_ELEMS<DT>, NW = NT / 32;
    extern __shared__ __align__(16) unsigned char smem[];
    uint4 *const ring = reinterpret_cast<uint4 *>(smem);
    using Shared = RowShared<NW, PARTS<OP>>;
    Shared &sh = *reinterpret_cast<Shared *>(ring + slots * U * NT);
    unsigned char *const lists = reinterpret_cast<unsigned char *>(&sh + 1);
    auto teacher = [&](int buf) {
        float *const f = reinterpret_cast<float *>(lists) + buf * 4 * teacher_k;
        return TeacherRow{reinterpret_cast<int *>(f), f + teacher_k, f + 2 * teacher_k, f + 3 * teacher_k};
    };
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int AHEAD = OP::TEACHER ? TEACHERS : 2;
    const int fixed = 3 * group + AHEAD;
    const float s2 = a.scale * LOG2E;
    pdl_enter();

    if (warp == NW && lane < fixed) {
        RowEntry e;
        e.state = ROW_END;
        const int64_t r = blockIdx.x + (int64_t)lane * gridDim.x;
        if (r < a.rows) {
            op.load(r, e);
            op.template settle<DT>(a, e);
        }
        sh.queue[lane] = e;
    }
    if (tid == 0) {
        for (int i = 0; i < slots; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], NW);
        }
        sh.published = fixed;
        sh.loading = 0;
        sh.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    volatile int *const failed = &sh.failed;
    volatile int *const published = &sh.published, *const loading = &sh.loading;

    // The barrier of row i: consumers, service warp and, of the teacher
    // warps, the row's own.  (The loader runs ahead by the slots alone.)
    auto row_barrier = [&](int i) {
        if constexpr (OP::TEACHER)
            bar_sync(1 + i % TEACHERS, NT + 64);
        else
            bar_sync(0, NT + 32);
    };
    // Batches of a row of nvec vectors, and how many of them are fetched twice.
    auto batches = [](int nvec) { return (nvec + U * NT - 1) / (U * NT); };
    auto twice = [&](int nb) { return OP::STATS && a.dx && nb > slots ? nb - slots : 0; };
    auto stat_of = [&](int i) {
        SoftStat t = lane < NW ? sh.part[i % PARTS<OP>][lane] : SoftStat{NEG_INF, 0.0f};
        if (*failed)
            t.l = __int_as_float(0x7fc00000);
        return soft_warp(t, s2);
    };

    if (warp == NW) {
        // ---- service warp
        unsigned taken = 0;  // link 1: the counter's value, in lane 0
        RowEntry got, ready;  // links 2 and 3, an entry in each of the first `group` lanes
        got.state = ready.state = ROW_END;
        got.r = ready.r = a.rows;
        for (int i = 0;; ++i) {
            const RowEntry e = sh.queue[i % ROW_Q];
            if (e.state == ROW_END)
                break;
            if (i % group == 0) {
                const int step = i / group;
                if (step >= 3) {
                    const int at = fixed + (step - 3) * group;
                    // (the loader may be behind on a run of ignored rows)
                    for (int n = 0; *loading + ROW_Q <= at + group && n < WAIT_TRIES && !*failed; ++n)
                        ;
                    if (lane < group)
                        sh.queue[(at + lane) % ROW_Q] = ready;
                    __threadfence_block();
                    __syncwarp();
                    if (lane == 0)
                        *published = at + group;
                }
                ready = got;
                if (ready.r < a.rows)
                    op.template settle<DT>(a, ready);
                got.state = ROW_END;
                got.r = a.rows;
                if (step >= 1) {
                    const int64_t r = (int64_t)fixed * gridDim.x + __shfl_sync(0xffffffffu, taken, 0) + lane;
                    if (lane < group && r < a.rows)
                        op.load(r, got);
                }
                if (lane == 0)
                    taken = atomicAdd(next, (unsigned)group);
            }
            row_barrier(i);
            const SoftStat t = OP::STATS ? stat_of(i) : SoftStat{};
            if (lane == 0)
                op.template write<DT>(a, e, t);
        }
        // the last CTA to finish leaves the counters as they were
        if (lane == 0) {
            __threadfence();
            if (atomicAdd(next + 1, 1u) == gridDim.x - 1) {
                next[0] = 0;
                next[1] = 0;
            }
        }
        return;
    }
    if (warp == NW + 1) {
        // ---- loader
        if (lane != 0)
            return;
        int slot = 0;
        uint32_t parity = 1;  // a fresh slot is empty
        for (int i = 0;; ++i) {
            for (int n = 0; *published <= i; ++n)
                if (n == WAIT_TRIES || *failed) {
                    *failed = 1;
                    return;
                }
            __threadfence_block();
            const int64_t r = sh.queue[i % ROW_Q].r;
            const int state = sh.queue[i % ROW_Q].state;
            *loading = i;
            if (state == ROW_END)
                break;
            if (state == ROW_OUT)
                continue;
            const T *row = static_cast<const T *>(a.x) + r * a.ld;
            const int h = head_elems<DT>(row, a.len), nvec = (a.len - h) / E;
            const int nb = batches(nvec), total = nb + twice(nb);
            row += h;
            for (int k = 0; k < total; ++k) {
                const int v0 = (k < nb ? k : k - nb) * U * NT;
                const int n = nvec - v0 < U * NT ? nvec - v0 : U * NT;
                mbar_wait(&sh.empty[slot], parity, failed);
                mbar_expect(&sh.full[slot], (uint32_t)n * 16u);
                bulk_load(ring + slot * U * NT, row + (int64_t)v0 * E, (uint32_t)n * 16u, &sh.full[slot]);
                if (++slot == slots) {
                    slot = 0;
                    parity ^= 1;
                }
            }
        }
        return;
    }
    if constexpr (OP::TEACHER) {
        if (warp > NW + 1) {
            // ---- teacher warp w: rows w, w + TEACHERS, ...
            const int w = warp - NW - 2;
            const TeacherRow list = teacher(w);
            for (int i = 0;; ++i) {
                // entries are visible a few rows ahead; walk to this warp's next
                const RowEntry e = sh.queue[i % ROW_Q];
                if (e.state == ROW_END)
                    break;
                if (i % TEACHERS != w)
                    continue;
                if (e.state == ROW_LIVE) {
                    const float Q = op.template prepare<DT>(a, e.r, list);
                    if (lane == 0)
                        sh.mass[w] = Q;
                }
                row_barrier(i);
                const SoftStat t = stat_of(i);
                const float Q = sh.mass[w];
                op.finish(a, e, t, list);
                if (a.dx && e.state == ROW_LIVE) {
                    const RowGrad g = op.template grad<DT>(a, e, t, Q);
                    bar_sync(1 + TEACHERS + w, NT + 32);
                    if (!g.zero)
                        op.template patch<DT>(a, e, g, list);
                }
                __syncwarp();
            }
            return;
        }
    }

    // ---- consumers
    const T *const x = static_cast<const T *>(a.x);
    T *const dx = static_cast<T *>(a.dx);
    int cslot = 0;  // slot of the next batch, and the phase it arrives in
    uint32_t cphase = 0;
    auto await_batch = [&]() { mbar_wait(&sh.full[cslot], cphase, failed); };
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

    for (int i = 0;; ++i) {
        const RowEntry e = sh.queue[i % ROW_Q];
        if (e.state == ROW_END)
            break;
        if (e.state == ROW_OUT) {
            row_barrier(i);
            if (dx)
                zero_row<DT>(dx + e.r * a.ldd, a.len, tid, NT);
            continue;
        }
        const T *const row = x + e.r * a.ld;
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

        SoftStat t{};
        const int first = cslot;
        if constexpr (OP::STATS) {
            SoftRun run;
            run.init();
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
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        run.template add<DT>(v[u], s2);
                } else {
#pragma unroll 1
                    for (int u = 0; u < U && u * NT < left; ++u) {
                        v[0] = src[u * NT];
                        run.raise(vec_max<DT>(v[0]), s2);
                        run.template add<DT>(v[0], s2);
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
            t = soft_warp(run.stat(), s2);
            if (lane == 0)
                sh.part[i % PARTS<OP>][warp] = t;
        }
        row_barrier(i);
        if (!dx)
            continue;
        if constexpr (OP::STATS)
            t = stat_of(i);
        const RowGrad g = op.template grad<DT>(a, e, t, OP::TEACHER ? sh.mass[i % TEACHERS] : 0.0f);
        T *const grow = dx + e.r * a.ldd;
        const bool aligned = ((uintptr_t)(grow + h) & 15u) == 0;
        auto emit = [&](int b, int slot) {
            const uint4 *src = ring + slot * U * NT + tid;
            const int j = h + (b * U * NT + tid) * E;
            const int left = nvec - b * U * NT - tid;
            uint4 v[U];
            if (g.zero) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u * NT < left)
                        store_vec<DT>(grow + j + u * NT * E, make_uint4(0, 0, 0, 0), aligned);
                release(slot);
            } else if (aligned && whole(b)) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    v[u] = src[u * NT];
                release(slot);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    *reinterpret_cast<uint4 *>(grow + j + u * NT * E) = vec_grad<DT>(v[u], g, j + u * NT * E);
            } else {
#pragma unroll 1
                for (int u = 0; u < U && u * NT < left; ++u)
                    store_vec<DT>(grow + j + u * NT * E, vec_grad<DT>(src[u * NT], g, j + u * NT * E), aligned);
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
        if (edge >= 0)
            store_elem<DT>(grow, edge, g.zero ? 0.0f : elem_grad<DT>(xe, g, edge));
        if constexpr (OP::TEACHER) {
            __threadfence_block();
            asm volatile("bar.arrive %0, %1;" ::"r"(1 + TEACHERS + i % TEACHERS), "n"(NT + 32) : "memory");
        }
    }
}

// ------------------------------------------------------------- short rows

constexpr int WARP_NT = 256;

// A warp per row, the row in registers (NV vectors per lane): rows too short
// for a CTA barrier each.  The next row's entry is fetched while this row is
// on its way.
template <int DT, class OP, int NV>
__global__ void __launch_bounds__(WARP_NT) warp_row_kernel(LogitRows a, OP op, int teacher_k)
{
    using T = typename Elem<DT>::T;
    constexpr int E = VEC_ELEMS<DT>;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *const f = reinterpret_cast<float *>(smem) + warp * 4 * teacher_k;
    const TeacherRow list{reinterpret_cast<int *>(f), f + teacher_k, f + 2 * teacher_k, f + 3 * teacher_k};
    const float s2 = a.scale * LOG2E;
    const T *const x = static_cast<const T *>(a.x);
    T *const dx = static_cast<T *>(a.dx);
    pdl_enter();

    const int64_t step = (int64_t)gridDim.x * (WARP_NT / 32);
    int64_t r = (int64_t)blockIdx.x * (WARP_NT / 32) + warp;
    RowEntry e{}, n{};
    if (r < a.rows) {
        op.load(r, n);
        op.template settle<DT>(a, n);
    }
    for (; r < a.rows; r += step) {
        e = n;
        T *const grow = dx + r * a.ldd;
        if (e.state == ROW_OUT) {
            if (r + step < a.rows) {
                op.load(r + step, n);
                op.template settle<DT>(a, n);
            }
            if constexpr (OP::TEACHER)
                op.finish(a, e, SoftStat{}, list);
            else if (lane == 0)
                op.template write<DT>(a, e, SoftStat{});
            if (dx)
                zero_row<DT>(grow, a.len, lane, 32);
            continue;
        }
        const T *const row = x + r * a.ld;
        const int h = head_elems<DT>(row, a.len), nvec = (a.len - h) / E;
        uint4 v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i * 32 + lane < nvec)
                v[i] = reinterpret_cast<const uint4 *>(row + h)[i * 32 + lane];
        int edge = -1;
        if (lane < h)
            edge = lane;
        else if (lane >= 8 && lane < 16 && h + nvec * E + lane - 8 < a.len)
            edge = h + nvec * E + lane - 8;
        float xe = 0.0f;
        if (edge >= 0)
            xe = load_elem<DT>(row, edge);
        if (r + step < a.rows)
            op.load(r + step, n);
        float Q = 0.0f;
        if constexpr (OP::TEACHER)
            Q = op.template prepare<DT>(a, r, list);

        SoftStat t{};
        if constexpr (OP::STATS) {
            float top = edge >= 0 ? xe : NEG_INF;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i * 32 + lane < nvec)
                    top = fmaxf(top, vec_max<DT>(v[i]));
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            SoftRun run;
            run.init();
            run.m = top;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i * 32 + lane < nvec)
                    run.template add<DT>(v[i], s2);
            if (edge >= 0)
                run.add(xe, s2);
            float l = run.l.x + run.l.y;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                l += __shfl_xor_sync(0xffffffffu, l, off);
            t = SoftStat{top, l};
            if constexpr (OP::TEACHER)
                op.finish(a, e, t, list);
            else if (lane == 0)
                op.template write<DT>(a, e, t);
        }
        if (r + step < a.rows)
            op.template settle<DT>(a, n);
        if (!dx)
            continue;
        const RowGrad g = op.template grad<DT>(a, e, t, Q);
        const bool aligned = ((uintptr_t)(grow + h) & 15u) == 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i * 32 + lane < nvec) {
                const int j = h + (i * 32 + lane) * E;
                store_vec<DT>(grow + j, g.zero ? make_uint4(0, 0, 0, 0) : vec_grad<DT>(v[i], g, j), aligned);
            }
        if (edge >= 0)
            store_elem<DT>(grow, edge, g.zero ? 0.0f : elem_grad<DT>(xe, g, edge));
        if constexpr (OP::TEACHER) {
            __syncwarp();
            if (!g.zero)
                op.template patch<DT>(a, e, g, list);
            __syncwarp();
        }
    }
}

// --------------------------------------------------------------- launchers

// Launch with dynamic shared memory and programmatic serialization (as
// launch_pdl).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_smem(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                            Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Longest row of the warp kernel.
constexpr size_t WARP_ROW_BYTES = 8192;

constexpr size_t SM_SMEM = 228 * 1024, CTA_SMEM = 227 * 1024, CTA_RESERVED = 1024;

template <int DT, class OP, int NT, int U>
int launch_row_kernel(const LogitRows &a, const OP &op, int per_sm, int teacher_k, cudaStream_t s, const DeviceInfo &di)
{
    Workspace ws;
    const int st = get_workspace(&ws);
    if (st != RED_OK)
        return st;
    constexpr int SERVICE = 32 * SERVICE_WARPS<OP>;
    constexpr size_t batch = (size_t)U * NT * 16;
    const size_t fixed = sizeof(RowShared<NT / 32, PARTS<OP>>) + (size_t)TEACHERS * 4 * 4 * teacher_k;
    size_t most = SM_SMEM / per_sm - CTA_RESERVED;
    most = most < CTA_SMEM ? most : CTA_SMEM;
    int slots = most > fixed ? (int)((most - fixed) / batch) : 0;
    slots = slots < ROW_MAX_SLOTS ? slots : ROW_MAX_SLOTS;
    if (slots < 2)
        slots = 2;
    const size_t smem = slots * batch + fixed;
    const auto kernel = row_kernel<DT, OP, NT, U>;
    static std::atomic<int> ready{0};
    if (!ready.load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)CTA_SMEM);
        if (e != cudaSuccess)
            return cuda_fail(e, "row kernel: shared memory");
        ready.store(1, std::memory_order_relaxed);
    }
    const int64_t cap = (int64_t)di.sms * per_sm;
    const unsigned grid = (unsigned)(a.rows < cap ? a.rows : cap);
    // Rows taken at a time: one where a CTA gets few rows (the last row taken
    // is what CTAs wait for at the end), more where rows are many.
    const int group = a.rows >= 32 * cap ? 4 : (a.rows >= 16 * cap ? 2 : 1);
    const cudaError_t e = launch_pdl_smem(kernel, grid, NT + SERVICE, smem, s, a, op, ws.tick, slots,
                                          group, teacher_k);
    count_launches(1);
    return cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "row kernel launch");
}

template <int DT, class OP, int NV>
int launch_warp_kernel(const LogitRows &a, const OP &op, int teacher_k, cudaStream_t s, const DeviceInfo &di)
{
    const auto kernel = warp_row_kernel<DT, OP, NV>;
    const size_t smem = (size_t)(WARP_NT / 32) * 4 * 4 * teacher_k;
    static std::atomic<int> ready{0};
    if (smem > 48 * 1024 && !ready.load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)CTA_SMEM);
        if (e != cudaSuccess)
            return cuda_fail(e, "warp row kernel: shared memory");
        ready.store(1, std::memory_order_relaxed);
    }
    int occ = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, (const void *)kernel, WARP_NT, smem);
    if (e != cudaSuccess || occ < 1)
        return cuda_fail(e, "warp row kernel: occupancy");
    const int64_t want = (a.rows + WARP_NT / 32 - 1) / (WARP_NT / 32), cap = (int64_t)di.sms * occ;
    e = launch_pdl_smem(kernel, (unsigned)(want < cap ? want : cap), WARP_NT, smem, s, a, op, teacher_k);
    count_launches(1);
    return cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "warp row kernel launch");
}

template <int DT, class OP>
int launch_rows_of(const LogitRows &a, const OP &op, int teacher_k, cudaStream_t s)
{
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != RED_OK)
        return st;
    const size_t bytes = (size_t)a.len * sizeof(typename Elem<DT>::T);
    if (bytes <= WARP_ROW_BYTES) {
        // vectors per lane of the longest interior
        const size_t nv = (bytes / 16 + 31) / 32;
        if (nv <= 2)
            return launch_warp_kernel<DT, OP, 2>(a, op, teacher_k, s, di);
        if (nv <= 8)
            return launch_warp_kernel<DT, OP, 8>(a, op, teacher_k, s, di);
        return launch_warp_kernel<DT, OP, 16>(a, op, teacher_k, s, di);
    }
    // Threads, vectors per thread and batch, and CTAs per SM, by row bytes.  A
    // CTA is busy with one row at a time, so short rows need several CTAs to
    // cover each other's barriers, and long ones a ring that holds a row and
    // the start of the next.  us, policy loss and gradient unless said:
    //                          512x4,1   256x4,2   256x4,3   128x4,4   128x4,6
    //   8192 x 65536 bf16          328       326       366       376       404
    //   4096 x 131072 bf16         358       434       460       478       491
    //   1000 x 32001 f32            52        58        60        61        64
    //   4096 x 16384 f32           106        99       105       109       114
    //   8192 x 16384 bf16          170       109       107       100       107
    //   16384 x 8192 bf16          262       139       133       110       106
    //   logprob 4096 x 50257 f16    65        56        54        56        56
    // (A loss with a gradient keeps its mapping when the gradient is not asked
    // for: the mapping sets the order of the sums.)
    if constexpr (!OP::GRADIENT)
        return launch_row_kernel<DT, OP, 256, 4>(a, op, 3, teacher_k, s, di);
    if (bytes > 98304)
        return launch_row_kernel<DT, OP, 512, 4>(a, op, 1, teacher_k, s, di);
    if (bytes > 49152)
        return launch_row_kernel<DT, OP, 256, 4>(a, op, 2, teacher_k, s, di);
    return launch_row_kernel<DT, OP, 128, 4>(a, op, bytes > 24576 ? 4 : 6, teacher_k, s, di);
}

template <class OP>
int launch_loss_rows(int dtype, const LogitRows &a, const OP &op, int teacher_k, cudaStream_t s)
{
    switch (dtype) {
    case RED_F32: return launch_rows_of<RED_F32>(a, op, teacher_k, s);
    case RED_F16: return launch_rows_of<RED_F16>(a, op, teacher_k, s);
    default: return launch_rows_of<RED_BF16>(a, op, teacher_k, s);
    }
}

// ------------------------------------------------------ totals over rows

constexpr int TOTAL_NT = 256, TOTAL_CTAS = 128, TOTAL_ROWS = 1024;

// N sums over the rows in 64 bits and a fixed order: each CTA sums its rows,
// the CTA that finishes last the CTAs' parts.  row(r, v) adds row r's terms.
template <int N, class ROW>
__device__ void total_rows(int64_t rows, ROW row, float *out, double *part, unsigned *tick)
{
    __shared__ double s[N][TOTAL_NT / 32];
    __shared__ bool s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto cta_total = [&](double (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            for (int off = 16; off > 0; off >>= 1)
                v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
            if (lane == 0)
                s[i][warp] = v[i];
        }
        __syncthreads();
        double t = 0.0;
        if (tid < N)
            for (int w = 0; w < TOTAL_NT / 32; ++w)
                t += s[tid][w];
        return t;  // total i in thread i
    };
    double v[N] = {};
    for (int64_t r = (int64_t)blockIdx.x * TOTAL_NT + tid; r < rows; r += (int64_t)gridDim.x * TOTAL_NT)
        row(r, v);
    double t = cta_total(v);
    if (gridDim.x == 1) {
        if (tid < N)
            out[tid] = (float)t;
        return;
    }
    if (tid < N)
        part[(int64_t)blockIdx.x * N + tid] = t;
    __threadfence();
    __syncthreads();
    if (tid == 0)
        s_last = atomicAdd(tick, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!s_last)
        return;
    __threadfence();
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = tid < gridDim.x ? __ldcg(part + (int64_t)tid * N + i) : 0.0;
    __syncthreads();
    t = cta_total(v);
    if (tid < N)
        out[tid] = (float)t;
    if (tid == 0)
        *tick = 0;
}

inline unsigned total_ctas(int64_t rows)
{
    const int64_t want = (rows + TOTAL_ROWS - 1) / TOTAL_ROWS;
    return (unsigned)(want < TOTAL_CTAS ? want : TOTAL_CTAS);
}

}  // namespace red
