// red_linear.cu -- log-probabilities of given tokens from hidden states h
// (rows x dim) and the vocabulary's weights w (vocab x dim), and their
// gradients, without the logits z = scale * h w^T ever being in memory.
//
//   forward    z tile by tile on the tensor cores; each tile leaves, per row,
//              its maximum and its sum of exponentials, without the target's; a
//              join adds that, from a product of its own in fp32, and makes lse
//              and logp.
//   backward   piece by piece of the vocabulary: z again, from it the gradient
//              by the logits,
//                  g_j = dlogp ([j = target] - p_j) + dlse p_j,  p_j = e^(z_j - lse),
//              in the inputs' 16-bit type, then the two products
//                  dh += g w_piece,   dw_piece = g^T h,
//              as tiles of one launch (both need nothing but g).
//
// Rows that do not take part are left out first: the others' hidden states are
// packed, which saves their share of the products and keeps what padded
// rows hold (NaN, say) out of dw.
#include <cuda.h>

#include "red_linear.cuh"
#include "red_loss.cuh"
#include "red_mma.cuh"
#include "red_prims.cuh"

namespace red {
namespace {

// Blocks of 64 of K whose products are summed by the tensor cores before the sum
// moves to fp32 registers (tiles of 256 x 256; of few rows, see Few).  The tensor cores'
// additions round toward zero, so a long sum drifts with its number of steps, four to a
// block, and lse with the logits: by -0.8e-6 on average at logits of a bell of width 1.5 (lse 11,
// dim 1024 to 8192; -1.9e-6 with 16 blocks), while 6144 x 4096 x 65536 bf16 takes 1675 us (1643
// with 16) and 2777 x 1024 x 50257 168 (162).  Against 64 bits logp is then off by 1.4e-7 to 2.0e-7 of its
// norm (300 rows; fp32 products of torch: 2.4e-7 at dim 1024, 5.8e-7 at 4096, 8.7e-7 at 8192).
// The gradients' logits, whose p are rounded to 16 bits, take 16.
// What the drift would do most harm to is the target's logit: the likelihood of a token that
// is all but certain is the distance of its logit from the others', and logits at the
// end of the range drift furthest.  That one is summed apart (dot_by_warp): a
// reading of N rows of both matrices.
constexpr int CHUNK = 8, CHUNK_GRAD = 16;
// Chunks of about CHUNK blocks, of equal length: 9 blocks are one chunk, not 8 and 1 (198 x 528 x 81709 30.6 us; 35.3 so).
int even_chunk(int blocks)
{
    const int n = (blocks + CHUNK / 2) / CHUNK;
    return n < 2 ? blocks : (blocks + n - 1) / n;
}
// The same of the gradients' sums, which are rounded to 16 bits at the end.  256 steps of terms of one sign are off by
// 3e-5 (measured: 1e-7 a step, of dw of 262144 rows -1.65e-3 in one run, three times f16's rounding, and -2e-5
// in runs of these); a sum of up to SHORT_PRODUCTS blocks, 1e-4, may be one run where rows are few.
constexpr int CHUNK_PRODUCTS = 64, SHORT_PRODUCTS = 256;
// Rows of tiles that are taken in turn along the vocabulary.
constexpr int BAND = 16;

struct TileAt {
    int m, n;
};
// Tile t of m_tiles x n_tiles: bands of BAND rows of tiles, in a band column by
// column, so that the tiles at work share both operands in L2.
__device__ __forceinline__ TileAt tile_at(int t, int m_tiles, int n_tiles)
{
    const int band = t / (BAND * n_tiles);
    const int in = t - band * BAND * n_tiles;
    const int high = min(BAND, m_tiles - band * BAND);
    return {band * BAND + in % high, in / high};
}

// Sum of the products of two rows (16-byte aligned) over `lanes` lanes: this one's share.
template <int DT>
__device__ __forceinline__ float dot_share(const uint16_t *h, const uint16_t *w, int64_t dim, int lane, int lanes)
{
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t vecs = dim / 8;
#pragma unroll 4
    for (int64_t i = lane; i < vecs; i += lanes) {
        const uint4 x = reinterpret_cast<const uint4 *>(h)[i], y = reinterpret_cast<const uint4 *>(w)[i];
        const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s[k] = fmaf(Elem<DT>::widen(u[k] & 0xffffu), Elem<DT>::widen(v[k] & 0xffffu), s[k]);
            s[k] = fmaf(Elem<DT>::widen(u[k] >> 16), Elem<DT>::widen(v[k] >> 16), s[k]);
        }
    }
    if (lane < dim % 8)
        s[0] = fmaf(Elem<DT>::widen(h[vecs * 8 + lane]), Elem<DT>::widen(w[vecs * 8 + lane]), s[0]);
    return (s[0] + s[1]) + (s[2] + s[3]);
}
__device__ __forceinline__ float sum_of_lanes(float v)
{
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Row r's hidden state times the weights of `target`, by a warp.
__device__ __forceinline__ float dot_by_warp(const LinearArgs &a, int64_t r, int64_t target, int lane)
{
    const uint16_t *h = static_cast<const uint16_t *>(a.hidden) + r * a.ldh;
    const uint16_t *w = static_cast<const uint16_t *>(a.weight) + target * a.ldw;
    return sum_of_lanes(a.dtype == RED_BF16 ? dot_share<RED_BF16>(h, w, a.dim, lane, 32)
                                            : dot_share<RED_F16>(h, w, a.dim, lane, 32));
}

// ------------------------------------------------------ rows that take part

constexpr int SCAN_NT = 1024, SCAN_ROWS = 8;

struct ScanArgs {
    LinearArgs in;
    const float *lse, *dlogp, *dlse;  // gradients only
    LinearWork w;
};

template <int NT, class V, class F>
__device__ __forceinline__ V block_fold(V v, V *sh, F f)
{
    for (int o = 16; o; o >>= 1)
        v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        sh[threadIdx.x / 32] = v;
    __syncthreads();
    v = sh[threadIdx.x % (NT / 32)];
    for (int o = NT / 64; o; o >>= 1)
        v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The largest coefficient of a call becomes this: the last bf16 below 2, where its
// rounding is finest relative to the value.  The gradient by the target's logit,
// -(1 - p) of the coefficient, is most of a row's gradient: with equal weights of 1 /
// 6144, which are 1.33 times a power of two, the errors of dh were 1.53 times those of
// rounding dh alone with a power of two as the unit, and are 1.15 times those with
// this.  In f16 it is 2^13 times that: a probability keeps all its digits down to 4e-9
// (6e-5 of 1.99 is where f16's steps stop shrinking: an even choice among 262144 was off by
// 0.4% each), and g, at most twice the largest coefficient, stays off the type's end.
constexpr float MOST = 1.9921875f;
__device__ __forceinline__ float most_of(int dtype) { return dtype == RED_F16 ? MOST * 8192.0f : MOST; }

// Which rows take part and, for the gradients, their coefficients, by a CTA of NT
// threads; the number of rows that take part.  f(place, row) for each; `writes`: to the
// workspace.  Thread t has rows t, t + NT, ... of a round, so that loads are of
// neighbours, and what a row needs is loaded at once, whether it takes part or not: one
// load after the other takes the latency of each, for every CTA of the gather.
template <int NT, int EACH>
struct ScanShared {
    int counts[EACH * (NT / 32)], all;
    float tops[32];
};
template <bool GRAD, int NT, int EACH, class F>
__device__ __forceinline__ int scan_rows(const ScanArgs &a, ScanShared<NT, EACH> &sh, bool writes, float &unit, F f)
{
    constexpr int WARPS = NT / 32, ROUND = NT * EACH;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    struct Row {
        int target;  // -1: outside the vocabulary
        float d, n;
    };
    auto load = [&](int64_t r) {
        Row row = {-1, 0.0f, 0.0f};
        if (r < a.in.rows) {
            const int64_t t = a.in.target[r];
            row.target = t >= 0 && t < a.in.vocab ? (int)t : -1;
            if constexpr (GRAD) {
                row.d = a.dlogp[r];
                row.n = a.dlse ? a.dlse[r] : 0.0f;
            }
        }
        return row;
    };
    auto takes_part = [&](const Row &row) {
        return row.target >= 0 && (!GRAD || !(row.d == 0.0f && row.n == 0.0f));
    };
    auto by_p = [&](const Row &row) { return (row.n - row.d) * a.in.scale; };
    // (a coefficient that is no number, or infinite, is its row's matter)
    auto size = [](float v) { return fabsf(v) < __builtin_huge_valf() ? fabsf(v) : 0.0f; };
    auto larger = [&](float top, const Row &row) {
        return takes_part(row) ? fmaxf(top, fmaxf(size(row.d * a.in.scale), size(by_p(row)))) : top;
    };
    Row row[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        row[i] = load(i * NT + tid);
    unit = 1.0f;
    if constexpr (GRAD) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            top = larger(top, row[i]);
#pragma unroll 4
        for (int64_t r = ROUND + tid; r < a.in.rows; r += NT)
            top = larger(top, load(r));
        top = block_fold<NT>(top, sh.tops, [](float x, float y) { return fmaxf(x, y); });
        if (top > 0.0f)
            unit = fminf(fmaxf(top, 1e-32f), 1e36f) / most_of(a.in.dtype);
    }
    const float inv = 1.0f / unit;
    int before = 0;
    for (int64_t r0 = 0; r0 < a.in.rows; r0 += ROUND) {
        if (r0 > 0) {
            __syncthreads();  // (the last round's counts have been read)
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                row[i] = load(r0 + i * NT + tid);
        }
        unsigned takes[EACH];  // by the warp's lanes
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            takes[i] = __ballot_sync(0xffffffffu, takes_part(row[i]));
            if (lane == 0)
                sh.counts[i * WARPS + warp] = __popc(takes[i]);
        }
        __syncthreads();
        if (warp == 0) {  // exclusive sums, in the order of the rows
            constexpr int MINE = EACH * WARPS / 32;
            int c[MINE], sum = 0;
#pragma unroll
            for (int k = 0; k < MINE; ++k) {
                c[k] = sum;
                sum += sh.counts[lane * MINE + k];
            }
            int upto = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o)
                    upto += v;
            }
#pragma unroll
            for (int k = 0; k < MINE; ++k)
                sh.counts[lane * MINE + k] = upto - sum + c[k];
            if (lane == 31)
                sh.all = upto;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int64_t r = r0 + i * NT + tid;
            if (r >= a.in.rows)
                break;
            const int at = before + sh.counts[i * WARPS + warp] + __popc(takes[i] & ((1u << lane) - 1u));
            const bool here = takes[i] >> lane & 1;
            if (writes)
                a.w.pos[r] = here ? at : -1;
            if (!here)
                continue;
            f(at, (int)r);
            if (writes) {
                a.w.idx[at] = (int)r;
                a.w.target[at] = row[i].target;
                if constexpr (GRAD) {
                    a.w.by_p[at] = by_p(row[i]) * inv;
                    a.w.lse2[at] = a.lse[r] * LOG2E;
                }
            }
        }
        before += sh.all;
    }
    if (writes && tid == 0) {
        a.w.head->live = before;
        a.w.head->unit = unit;
    }
    return before;
}

template <bool GRAD>
__global__ void __launch_bounds__(SCAN_NT) linear_scan_kernel(const ScanArgs a)
{
    pdl_enter();
    __shared__ ScanShared<SCAN_NT, SCAN_ROWS> sh;
    float unit;
    scan_rows<GRAD, SCAN_NT, SCAN_ROWS>(a, sh, true, unit, [](int, int) {});
}

// g at the target of packed row r (`row` of the input), by a warp: from a logit of its own.
// 1 - p of a token that is all but certain is as exact as lse.
__device__ __forceinline__ void write_at_target(const ScanArgs &a, int64_t r, int64_t row, float unit, int lane)
{
    const float z = dot_by_warp(a.in, row, a.in.target[row], lane);
    if (lane == 0) {
        const float d = a.dlogp[row], n = a.dlse ? a.dlse[row] : 0.0f;
        const float p = expf(fmaf(z, a.in.scale, -a.lse[row]));
        a.w.at_target[r] = (d + (n - d) * p) * a.in.scale * (1.0f / unit);
    }
}

// Row `row` of the hidden states (-1: zeros) to packed row r, by a warp.
__device__ __forceinline__ void pack_row(const void *hidden, int64_t dim, int64_t ldh, const LinearWork &w, int64_t r,
                                         int row, int lane)
{
    const int64_t vecs = dim / 8;
    const int tail = (int)(dim % 8);
    uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(w.hidden) + r * w.ld);
    const uint16_t *from = row >= 0 ? static_cast<const uint16_t *>(hidden) + row * ldh : nullptr;
    const uint4 *v = reinterpret_cast<const uint4 *>(from);
    int64_t i = lane;
    for (; i + 96 < vecs && from; i += 128) {
        const uint4 v0 = v[i], v1 = v[i + 32], v2 = v[i + 64], v3 = v[i + 96];
        to[i] = v0;
        to[i + 32] = v1;
        to[i + 64] = v2;
        to[i + 96] = v3;
    }
    for (; i < vecs; i += 32)
        to[i] = from ? v[i] : make_uint4(0, 0, 0, 0);
    if (lane < tail)
        reinterpret_cast<uint16_t *>(to)[vecs * 8 + lane] = from ? from[vecs * 8 + lane] : (uint16_t)0;
}

// The hidden states of the rows that take part, packed; a warp per row.  Zeros
// up to a whole tile behind them.
template <bool GRAD>
__global__ void __launch_bounds__(256) linear_pack_kernel(const ScanArgs a)
{
    pdl_enter();
    const int live = a.w.head->live;
    const int64_t end = ((int64_t)live + TILE - 1) / TILE * TILE;
    const int lane = threadIdx.x % 32;
    for (int64_t r = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; r < end; r += (int64_t)gridDim.x * 8) {
        const int row = r < live ? a.w.idx[r] : -1;
        pack_row(a.in.hidden, a.in.dim, a.in.ldh, a.w, r, row, lane);
        if (GRAD && row >= 0)
            write_at_target(a, r, row, a.w.head->unit, lane);
    }
}

// Of few rows, at most half as many as there are columns of the piece: g in two parts of 16 bits, packed row r's in
// columns r and r + few / 2, whose packed row is r's again.  A gradient by few logits is most of the results'
// error when it is rounded to 16 bits once: of one row, every value of dw is a single product (1 to 3 rows of f16:
// 1.1 to 1.6 times the error that rounding the results leaves; not to be seen beside it so).
__device__ __forceinline__ bool two_parts(int live, int few) { return live <= few / 2; }

// Both for up to a few thousand rows, in one launch: every CTA does the scan for itself,
// and packs eight rows.
constexpr int GATHER_ROWS = 4096;
template <bool GRAD, int EACH>
__global__ void __launch_bounds__(256) linear_gather_kernel(const ScanArgs a)
{
    pdl_enter();
    __shared__ ScanShared<256, EACH> sh;
    __shared__ int row_of[8], twin_of[8];
    const bool writes = blockIdx.x == 0;
    const int first_packed = blockIdx.x * 8;
    if (threadIdx.x < 8)
        row_of[threadIdx.x] = twin_of[threadIdx.x] = -1;
    float unit;
    const int live = scan_rows<GRAD, 256, EACH>(a, sh, writes, unit, [&](int at, int r) {
        if (at >= first_packed && at < first_packed + 8)
            row_of[at - first_packed] = r;
        const int twin = at + a.w.few / 2 - first_packed;
        if (GRAD && twin >= 0 && twin < 8)
            twin_of[twin] = r;
    });
    __syncthreads();
    const int64_t r = first_packed + threadIdx.x / 32;
    if (r >= (live + TILE - 1) / TILE * TILE)
        return;
    const int row = GRAD && r >= live && two_parts(live, a.w.few) ? twin_of[threadIdx.x / 32] : row_of[threadIdx.x / 32];
    pack_row(a.in.hidden, a.in.dim, a.in.ldh, a.w, r, row, threadIdx.x % 32);
    if (GRAD && row >= 0 && r < live)
        write_at_target(a, r, row, unit, threadIdx.x % 32);
}

// --------------------------------------------------------------- logit tiles

struct LogitArgs {
    CUtensorMap h, w, g;
    LinearWork work;
    int v0, n_tiles;   // columns of the vocabulary: the first, and tiles from it on
    int vocab, k_blocks;
    int chunk;         // blocks of K to a run of sums
    float s2;          // scale * log2(e)
};

// One warp's 32 rows x 128 columns of a product in fp32 registers: the sums of
// the chunks of `each` blocks.  Whether they are right: after a wait that ran out they are whatever
// tensor memory held (and what is made of them has to become NaN; filling them
// here costs the registers of a second set).
__device__ __forceinline__ bool take_sums(float (&z)[HALF], MmaBarriers &b, AccPos &acc, int blocks, int each,
                                          uint32_t lanes, int half, uint32_t (&empty)[2])
{
    bool ok = true;
    for (int k = 0; k < blocks; k += each) {
        ok &= mbar_wait(&b.acc_full[acc.slot], acc.phase, &b.failed, 0);
        tmem_after();
        const uint32_t from = b.tmem + lanes + acc.slot * TILE + half * HALF;
        if (k == 0) {
#pragma unroll
            for (int i = 0; i < HALF; i += 16)
                tmem_load16(from + i, reinterpret_cast<uint32_t *>(z + i));
            tmem_wait();
        } else {
#pragma unroll
            for (int i = 0; i < HALF; i += 32) {
                uint32_t v[32];
                tmem_load16(from + i, v);
                tmem_load16(from + i + 16, v + 16);
                tmem_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    z[i + j] += __uint_as_float(v[j]);
            }
        }
        tmem_before();
        __syncwarp();
        if (threadIdx.x % 32 == 0)
            arrive_at(empty[acc.slot]);
        acc.next();
    }
    return ok;
}

// What the exponents of terms under the maximum m are relative to: m * s2, rounded, and the factor that makes their
// sum relative to m itself, 2^(the rounding).  Maxima of tiles differ by the size of the logits, and their products'
// roundings would be in every term of one of them: of logits near 20, 1e-6.
struct Base {
    float off;

    __device__ __forceinline__ Base(float m, float s2) { off = m == NEG_INF ? 0.0f : __fmul_rn(m, s2); }
    __device__ __forceinline__ float factor(float m, float s2) const
    {
        return m == NEG_INF ? 1.0f : ex2(-fmaf(m, s2, -off));
    }
};

// Two floats as 16-bit values, the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if constexpr (DT == RED_BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// GRAD: g of the tile to `piece`; else the tile's statistics to `part`.
template <int DT, bool GRAD>
__global__ void __launch_bounds__(MMA_THREADS, 1) linear_logits_kernel(const __grid_constant__ LogitArgs a)
{
    extern __shared__ unsigned char raw[];
    __shared__ MmaBarriers b;
    unsigned char *const ring = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = cluster_rank();
    mma_begin(b, warp, lane);
    pdl_enter();
    const int live = a.work.head->live;
    const int m_tiles = (live + TILE - 1) / TILE;
    const int tiles = m_tiles * a.n_tiles;
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

    auto job = [&](TileAt at) {
        return TileJob{&a.h, &a.w, at.m * TILE, a.v0 + at.n * TILE, 0, 0, a.k_blocks, true, true};
    };
    if (warp < 4)
        fewer_registers();
    if (warp == 0 && lane == 0) {
        RingPos<> pos;
        for (int t = pair; t < tiles; t += pairs)
            if (!copy_tile(job(tile_at(t, m_tiles, a.n_tiles)), b, ring, pos, rank)) {
                drain_copies(b, pos, rank);
                break;
            }
    } else if (warp == 1 && rank == 0) {
        const bool issues = elect_one();
        RingPos<> pos;
        AccPos acc;
        const uint32_t idesc = instruction_desc(DT == RED_BF16, true, true);
        for (int t = pair; t < tiles; t += pairs)
            if (!multiply_tile<true>(job(tile_at(t, m_tiles, a.n_tiles)), b, ring, pos, acc, idesc, a.chunk,
                                     issues)) {
                drain_products(b, issues);
                break;
            }
    } else if (warp >= 4) {
        more_registers();  // the sums of a tile take 128 per thread
        AccPos acc;
        const int group = warp % 4, half = (warp - 4) / 4;
        uint32_t empty[2] = {leader_addr(&b.acc_empty[0]), leader_addr(&b.acc_empty[1])};
        unsigned char *const staging = ring + STAGES * STAGE_BYTES + (warp - 4) * STAGING_BYTES;
        for (int t = pair; t < tiles; t += pairs) {
            const TileAt at = tile_at(t, m_tiles, a.n_tiles);
            const int row = at.m * TILE + rank * HALF + group * 32 + lane;
            const int col = a.v0 + at.n * TILE + half * HALF;
            const bool takes = row < live;
            const int target = takes ? a.work.target[row] - col : -1;
            const bool tail = col + HALF > a.vocab;
            float z[HALF];
            // (the row's coefficients are on their way while the products are)
            float gt = 0.0f, cp = 0.0f, lse2 = 0.0f;
            if (GRAD && takes)
                gt = a.work.at_target[row], cp = a.work.by_p[row], lse2 = a.work.lse2[row];
            const bool ok = take_sums(z, b, acc, a.k_blocks, a.chunk, (uint32_t)(group * 32) << 16, half, empty);
            constexpr float NOTHING = __builtin_nanf("");
            if constexpr (!GRAD) {
                if (tail) {
#pragma unroll
                    for (int i = 0; i < HALF; ++i)
                        if (col + i >= a.vocab)
                            z[i] = NEG_INF;
                }
                if (__any_sync(0xffffffffu, (unsigned)target < (unsigned)HALF)) {
#pragma unroll
                    for (int i = 0; i < HALF; ++i)
                        z[i] = i == target ? NEG_INF : z[i];  // (the join adds it)
                }
                float m = NEG_INF;
#pragma unroll
                for (int i = 0; i < HALF; i += 2)
                    m = fmaxf(m, fmaxf(z[i], z[i + 1]));
                const Base base(m, a.s2);
                float l[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < HALF; ++i)
                    l[i % 4] += ex2(fmaf(z[i], a.s2, -base.off));
                if (takes)
                    a.work.part[(int64_t)row * a.work.slots + (at.n * 2 + half)] =
                        make_float2(m, ok ? ((l[0] + l[1]) + (l[2] + l[3])) * base.factor(m, a.s2) : NOTHING);
            } else {
                cp = ok ? cp : NOTHING;
                gt = ok ? gt : NOTHING;
                const bool here = __any_sync(0xffffffffu, (unsigned)target < (unsigned)HALF);
#pragma unroll
                for (int i = 0; i < HALF; ++i)
                    z[i] = cp * ex2(fmaf(z[i], a.s2, -lse2));
                if (here) {
#pragma unroll
                    for (int i = 0; i < HALF; ++i)
                        z[i] = i == target ? gt : z[i];
                }
                if (__any_sync(0xffffffffu, !takes)) {
                    // rows behind the last one: their logits are 0, or NaN where a weight is -inf
#pragma unroll
                    for (int i = 0; i < HALF; ++i)
                        z[i] = takes ? z[i] : 0.0f;
                }
                if (tail) {
#pragma unroll
                    for (int i = 0; i < HALF; ++i)
                        if (col + i >= a.vocab)
                            z[i] = 0.0f;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    // 32 rows of 64 columns through shared memory, 16-byte units swizzled as the map says
                    unsigned char *const box = staging + c * BOX_BYTES;
                    if (lane == 0)
                        store_read<1>();
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const float *v = z + c * 64 + u * 8;
                        *reinterpret_cast<uint4 *>(box + lane * 128 + ((u ^ (lane & 7)) * 16)) =
                            make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]),
                                       pack2<DT>(v[6], v[7]));
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store(&a.g, at.n * TILE + half * HALF + c * 64, at.m * TILE + rank * HALF + group * 32,
                                  box);
                        store_commit();
                    }
                }
            }
        }
        if (GRAD && lane == 0)
            store_done();
    }
    __syncwarp();
    mma_end(b, warp);
}

__device__ __forceinline__ float max_of_warp(float v)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// ----------------------------------------------------------- join of the parts

// (maximum, sum) pairs of a row's tiles to its lse and logp: a warp per row, or a CTA
// where rows are few.
struct Pair {
    float m, l;
    __device__ __forceinline__ void join(float om, float ol, float s2)
    {
        const float top = fmaxf(m, om);
        const float ref = top == NEG_INF ? 0.0f : top;
        l = l * ex2((m - ref) * s2) + ol * ex2((om - ref) * s2);
        m = top;
    }
    __device__ __forceinline__ void join_lanes(float s2)
    {
        const float top = max_of_warp(m);
        l = sum_of_lanes(l * ex2((m - (top == NEG_INF ? 0.0f : top)) * s2));
        m = top;
    }
};

template <int LANES>
__global__ void __launch_bounds__(256)
    linear_join_kernel(const LinearArgs a, const LinearWork w, int64_t slots, float s2, float *logp, float *lse)
{
    pdl_enter();
    __shared__ float2 warps[8];
    __shared__ float dots[8];
    constexpr int GROUPS = 256 / LANES;
    const int lane = threadIdx.x % LANES;
    for (int64_t r = (int64_t)blockIdx.x * GROUPS + threadIdx.x / LANES; r < a.rows; r += (int64_t)gridDim.x * GROUPS) {
        const int64_t target = a.target[r];
        const bool takes = target >= 0 && target < a.vocab;
        if (!takes) {  // (a CTA's row is the same for all its threads)
            if (lane == 0)
                logp[r] = lse[r] = 0.0f;
            continue;
        }
        const float2 *part = w.part + (w.few ? r : (int64_t)w.pos[r]) * w.slots;
        Pair p = {NEG_INF, 0.0f};
#pragma unroll 4
        for (int64_t i = lane; i < slots; i += LANES) {
            const float2 o = part[i];
            p.join(o.x, o.y, s2);
        }
        p.join_lanes(s2);
        float z;  // the target's product
        if constexpr (LANES > 32) {
            const uint16_t *hr = static_cast<const uint16_t *>(a.hidden) + r * a.ldh;
            const uint16_t *wr = static_cast<const uint16_t *>(a.weight) + target * a.ldw;
            z = sum_of_lanes(a.dtype == RED_BF16 ? dot_share<RED_BF16>(hr, wr, a.dim, lane, LANES)
                                                 : dot_share<RED_F16>(hr, wr, a.dim, lane, LANES));
            __syncthreads();
            if (lane % 32 == 0) {
                warps[lane / 32] = make_float2(p.m, p.l);
                dots[lane / 32] = z;
            }
            __syncthreads();
            p = {NEG_INF, 0.0f};
            if (lane % 32 < LANES / 32)
                p = {warps[lane % 32].x, warps[lane % 32].y};
            p.join_lanes(s2);
            z = 0.0f;
#pragma unroll
            for (int k = 0; k < LANES / 32; ++k)
                z += dots[k];
        } else {
            z = dot_by_warp(a, r, target, lane);
        }
        if (lane == 0) {
            const float off = z - p.m;  // (a NaN goes on; +inf, and only +inf, is one below)
            float lp, norm;
            if (off >= 0.0f) {
                lp = log1pf(p.l * ex2(-off * s2));
                norm = fmaf(z, a.scale, lp) + (z - z);
                lp = (z - z) - lp;
            } else {
                const float all = logf(p.l + ex2(off * s2));
                norm = fmaf(p.m, a.scale, all);
                lp = fmaf(off, a.scale, -all);
            }
            logp[r] = lp;
            lse[r] = norm;
        }
    }
}

// ------------------------------------------------------------ few rows

// Up to 128 rows: the weights' way through memory is what bounds a call, and tiles
// of 256 rows x 256 columns would load as much of (packed, mostly empty) rows as of
// weights, 76 at a time.  Here the weights are the operand with 128 rows, the hidden
// states the one with ROWS = 16, 32, 64 or 128, and each CTA takes an equal share of the
// vocabulary in tiles of equal height (up to 128), so that all SMs stream weights to the
// end; a tile is one copy per block of K, whatever its height.  Forward, us, with tiles of
// 256 x 256 / of 128 with an end in boxes of 16 / of equal height / the rows unpacked / the
// products issued by an elected lane, from several sums (as it is): 1 x 2048 x 65536 61, 58, 52, 47, 46;
// 16 x 4096 x 50257 -, 88, 75, 69, 67.  The
// stages in flight are not what bounds it (4 of 18 KB instead of 11 cost 8%, 7 cost 2%),
// nor is the rows' distance in memory; 128 bytes of each of many rows at a time come at 5.4
// to 5.7 TB/s where one stream of all rows comes at 6.5.
constexpr int FEW_ROWS = 128, FEW_THREADS = 256, FEW_MAX_CTAS = 512;

template <int ROWS, bool GRAD>
struct Few {
    static constexpr int STAGE = OPERAND_BYTES + ROWS * BLOCK_K * 2;
    static constexpr int N = 212992 / STAGE < 12 ? 212992 / STAGE : 12;  // stages
    static constexpr size_t SMEM = (size_t)N * STAGE + 1024;
    // The blocks of a chunk go to ACCS sums in turn, which meet in fp32 registers: 8 to 16 steps that round toward
    // zero in a row instead of the 64 of one sum of 16 blocks.  One row's log-probability stands alone, and was
    // off by up to 2.2e-6 of itself (1 x 1024 x 32001; 6.2e-7 so).  The gradients' logits, whose p are rounded to 16 bits,
    // have one sum: their weights may come from L2, and the epilogue is then what a tile waits for (a step of 100 x
    // 1024 x 32001 91 us with two sums, 88 so).
    static constexpr int ACCS = GRAD ? 1 : ROWS <= 32 ? 8 : 256 / ROWS;
    static constexpr int CHUNK = GRAD || ROWS <= 64 ? 16 : 8;
    static constexpr int COLUMNS = 2 * ACCS * ROWS;  // of tensor memory
    struct Shared {
        uint64_t full[N], empty[N], acc_full[2], acc_empty[2], drain;
        uint32_t tmem;
        int failed;
        float2 stats[4][ROWS];
        int target[ROWS];
        float4 coefs[ROWS];  // of p, g at the target, lse
    };
};

struct FewArgs {
    CUtensorMap h, w;  // boxes of 64 x ROWS, 64 x height
    LinearWork work;
    int vocab, k_blocks;
    int height, tiles;  // of each CTA
    float s2;
    // Forward: the rows as they are, `rows` of them with these targets.  One that takes no part is no
    // more than a column that nobody reads; the gradients take packed rows (its NaN would reach dw).
    const int64_t *targets;
    int rows;
};

// Sums over the warp of 32 (or the first 16) values per lane: lane i gets the i-th.
template <int N>
__device__ __forceinline__ float sums_of_warp(float *v, int lane)
{
    static_assert(N == 16 || N == 32, "");
    if constexpr (N == 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
    }
#pragma unroll
    for (int o = N / 2; o; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0];
}

template <int DT, bool GRAD, int ROWS>
__global__ void __launch_bounds__(FEW_THREADS, 1) linear_few_kernel(const __grid_constant__ FewArgs a)
{
    using F = Few<ROWS, GRAD>;
    extern __shared__ unsigned char raw[];
    __shared__ typename F::Shared b;
    unsigned char *const ring = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;  // (the same for a warp)
    if (threadIdx.x == 0) {
        for (int i = 0; i < F::N; ++i) {
            mbar_init(&b.full[i], 1);
            mbar_init(&b.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.acc_full[i], 1);
            mbar_init(&b.acc_empty[i], 4);
        }
        mbar_init(&b.drain, 1);
        b.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2)
        tmem_alloc_alone<F::COLUMNS>(&b.tmem);
    pdl_enter();
    const int live = GRAD ? a.work.head->live : a.rows;
    for (int r = threadIdx.x; r < ROWS; r += FEW_THREADS) {
        const bool takes = r < live;
        if (GRAD) {
            b.target[r] = takes ? a.work.target[r] : -1;
        } else {
            const int64_t t = takes ? a.targets[r] : -1;
            b.target[r] = t >= 0 && t < a.vocab ? (int)t : -1;
        }
        if (GRAD)
            b.coefs[r] = takes ? make_float4(a.work.by_p[r], a.work.at_target[r], a.work.lse2[r], 0.0f)
                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    tmem_before();
    __syncthreads();
    tmem_after();
    // this CTA's columns of the vocabulary
    const int begin = blockIdx.x * a.tiles * a.height, end = min(begin + a.tiles * a.height, a.vocab);

    if (live == 0) {
        // nothing takes part, and nothing reads the piece
    } else if (warp == 0 && lane == 0) {
        RingPos<F::N> pos;
        bool ok = true;
        for (int v = begin; v < end && ok; v += a.height)
            for (int k = 0; k < a.k_blocks; ++k) {
                if (!mbar_wait(&b.empty[pos.stage], pos.phase ^ 1, &b.failed, 0)) {
                    ok = false;
                    break;
                }
                uint64_t *const bar = &b.full[pos.stage];
                mbar_expect(bar, (uint32_t)((a.height + ROWS) * BLOCK_K * 2));
                unsigned char *const at = ring + pos.stage * F::STAGE;
                tma_load_alone(at, &a.w, k * BLOCK_K, v, bar);
                tma_load_alone(at + OPERAND_BYTES, &a.h, k * BLOCK_K, 0, bar);
                pos.next();
            }
        if (!ok)
            for (int k = 0; k < F::N; ++k)
                for (int n = 0; n < 65536 && !mbar_try(&b.full[k], k < pos.stage ? pos.phase : pos.phase ^ 1); ++n) {
                }
    } else if (warp == 1) {
        // All lanes wait and one issues: what the products take is then known to be the same for the warp, and a block
        // of K is not bound by one thread's moving it there (1 x 2048 x 65536 with eight sums 50.3 -> 45.0 us).
        const bool issues = elect_one();
        RingPos<F::N> pos;
        AccPos acc;
        bool ok = true;
        const uint32_t idesc = instruction_desc(DT == RED_BF16, true, true, HALF, ROWS);
        for (int v = begin; v < end && ok; v += a.height)
            for (int k0 = 0; k0 < a.k_blocks && ok; k0 += F::CHUNK) {
                if (!agreed(mbar_wait(&b.acc_empty[acc.slot], acc.phase ^ 1, &b.failed, 0))) {
                    ok = false;
                    break;
                }
                tmem_after();
                for (int k = k0; k < min(k0 + F::CHUNK, a.k_blocks); ++k) {
                    if (!agreed(mbar_wait(&b.full[pos.stage], pos.phase, &b.failed, 0))) {
                        ok = false;
                        break;
                    }
                    tmem_after();
                    const unsigned char *at = ring + pos.stage * F::STAGE;
                    const uint32_t d = b.tmem + (acc.slot * F::ACCS + (k - k0) % F::ACCS) * ROWS;
                    const uint64_t da = operand_desc(at, true), db = operand_desc(at + OPERAND_BYTES, true);
                    if (issues) {
#pragma unroll
                        for (int s = 0; s < BLOCK_K / 16; ++s)
                            mma_alone(d, da + s * step_k(true), db + s * step_k(true), idesc, k - k0 >= F::ACCS || s > 0);
                        mma_commit_alone(&b.empty[pos.stage]);
                    }
                    pos.next();
                }
                if (ok && issues)
                    mma_commit_alone(&b.acc_full[acc.slot]);
                acc.next();
            }
        if (!ok) {
            if (issues)
                mma_commit_alone(&b.drain);
            for (int n = 0; n < 65536 && !mbar_try(&b.drain, 0); ++n) {
            }
        }
    } else if (warp >= 4) {
        constexpr int GROUP = ROWS < 32 ? ROWS : 32, GROUPS = ROWS / GROUP;
        const int part = warp - 4;
        AccPos acc;
        float m[GROUPS], l[GROUPS];  // lane i: of rows g * 32 + i
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
            m[g] = NEG_INF, l[g] = 0.0f;
        for (int v0 = begin; v0 < end; v0 += a.height) {
            const int first = v0 + part * 32, v = first + lane;
            const int stop = min(v0 + a.height, end);  // (rows of the tile behind it hold what was there before)
            const bool valid = v < stop;
            float z[ROWS];
            bool ok = true;
            for (int k = 0; k < a.k_blocks; k += F::CHUNK) {
                ok &= mbar_wait(&b.acc_full[acc.slot], acc.phase, &b.failed, 0);
                tmem_after();
                uint32_t from = b.tmem + ((uint32_t)(part * 32) << 16) + acc.slot * F::ACCS * ROWS;
                for (int n = 0; n < min(F::ACCS, a.k_blocks - k); ++n, from += ROWS) {
                    if (k == 0 && n == 0) {
#pragma unroll
                        for (int i = 0; i < ROWS; i += 16)
                            tmem_load16(from + i, reinterpret_cast<uint32_t *>(z + i));
                        tmem_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < ROWS; i += 16) {
                            uint32_t x[16];
                            tmem_load16(from + i, x);
                            tmem_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                z[i + j] += __uint_as_float(x[j]);
                        }
                    }
                }
                tmem_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&b.acc_empty[acc.slot]);
                acc.next();
            }
            const float fine = ok ? 0.0f : __builtin_nanf("");
            if constexpr (!GRAD) {
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    // a target among this warp's columns
                    const int t = lane < GROUP ? b.target[g * 32 + lane] - first : -1;
                    unsigned here = __ballot_sync(0xffffffffu, t >= 0 && t < 32 && first + t < stop);
                    while (here) {  // (the join adds it)
                        const int i = __ffs(here) - 1;
                        here &= here - 1;
                        const bool mine = lane == __shfl_sync(0xffffffffu, t, i);
#pragma unroll
                        for (int j = 0; j < GROUP; ++j)
                            z[g * 32 + j] = mine && j == i ? NEG_INF : z[g * 32 + j];
                    }
                    float e[GROUP];
                    float top = NEG_INF;  // of row `lane`
#pragma unroll
                    for (int j = 0; j < GROUP; ++j) {
                        const float x = valid ? z[g * 32 + j] : NEG_INF;
                        const float most = max_of_warp(x);
                        e[j] = ex2(fmaf(x, a.s2, -Base(most, a.s2).off));
                        top = j == lane ? most : top;
                    }
                    const float sum = sums_of_warp<GROUP>(e, lane) * Base(top, a.s2).factor(top, a.s2) + fine;
                    Pair p = {m[g], l[g]};
                    p.join(top, sum, a.s2);
                    m[g] = p.m, l[g] = p.l;
                }
            } else {
                uint4 *to = reinterpret_cast<uint4 *>(a.work.piece) + (int64_t)v * (ROWS / 8);
                auto logit_gradients = [&](int i, float (&x)[8]) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 c = b.coefs[i + j];
                        const float g = v == b.target[i + j] ? c.y : c.x * ex2(fmaf(z[i + j], a.s2, -c.z));
                        // (rows behind the last one: their logits are 0, or NaN where a weight is -inf)
                        x[j] = (i + j < live ? g : 0.0f) + fine;
                    }
                };
                auto pack8 = [](const float (&x)[8]) {
                    return make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]),
                                      pack2<DT>(x[6], x[7]));
                };
                if (two_parts(live, ROWS)) {
#pragma unroll
                    for (int i = 0; i < ROWS / 2; i += 8) {
                        float x[8];
                        logit_gradients(i, x);
                        const uint4 whole = pack8(x);
                        const uint32_t u[4] = {whole.x, whole.y, whole.z, whole.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {  // what that leaves
                            x[2 * k] -= Elem<DT>::widen(u[k] & 0xffffu);
                            x[2 * k + 1] -= Elem<DT>::widen(u[k] >> 16);
                        }
                        if (valid) {
                            to[i / 8] = whole;
                            to[i / 8 + ROWS / 16] = pack8(x);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < ROWS; i += 8) {
                        float x[8];
                        logit_gradients(i, x);
                        if (valid)
                            to[i / 8] = pack8(x);
                    }
                }
            }
        }
        if constexpr (!GRAD) {
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
                if (lane < GROUP)
                    b.stats[part][g * 32 + lane] = make_float2(m[g], l[g]);
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const int r = threadIdx.x - 128;
            if (r < live) {
                Pair p = {NEG_INF, 0.0f};
                for (int w = 0; w < 4; ++w)
                    p.join(b.stats[w][r].x, b.stats[w][r].y, a.s2);
                a.work.part[(int64_t)r * a.work.slots + blockIdx.x] = make_float2(p.m, p.l);
            }
        }
    }
    __syncwarp();
    tmem_before();
    __syncthreads();
    tmem_after();
    if (warp == 2)
        tmem_free_alone<F::COLUMNS>(b.tmem);
}

// ------------------------------------------------------- products with weights

struct ProductArgs {
    CUtensorMap g_h;    // piece (dh: A): boxes of 64 of the vocabulary x 128 rows, of few rows 64 rows x 64
    CUtensorMap w_n;    // weights, along dim: boxes of 64 x 64                  (dh: B)
    CUtensorMap g_w;    // piece (dw: A): boxes of 64 of the vocabulary x 64 rows, of few rows 64 rows x 128
    CUtensorMap h_n;    // packed hidden states, along dim: boxes of 64 x 64     (dw: B)
    CUtensorMap dh, dw; // results: boxes of 32 x 32 fp32, 64 x 32 16-bit
    LinearWork work;
    int v0, v_count;    // the piece: first column of the vocabulary, columns
    int n_tiles;        // along dim
    int splits;         // of dh, along the vocabulary
    bool few;           // the piece lies along the rows
    int first;          // dh: store (1) or add (0)
    uint16_t *dweight;  // dw's memory, for the end of rows that do not end on 16 bytes
    int64_t lddw;
    int dim, vocab;
    int with_dh, with_dw;
};

// WIDTH columns of a warp's 32 rows of a product, 128 bytes of each row, to memory.
template <bool DH>
constexpr int PRODUCT_WIDTH = DH ? 32 : 64;
template <int DT, bool DH>
__device__ __forceinline__ void store_columns(const ProductArgs &a, const float *v, int row, int col, int c, float unit,
                                              unsigned char *staging, int lane)
{
    constexpr int WIDTH = PRODUCT_WIDTH<DH>;
    if (!DH && a.dim % 8 != 0 && col + c < a.dim && col + c + WIDTH > a.dim) {
        // (a map's box ends on 16 bytes, here beyond the row)
        const int64_t r = (int64_t)a.v0 + row + lane;
        if (r < a.vocab) {
#pragma unroll
            for (int i = 0; i < WIDTH; ++i)
                if (col + c + i < a.dim)
                    a.dweight[r * a.lddw + col + c + i] = (uint16_t)pack2<DT>(v[i] * unit, 0.0f);
        }
        // An empty group in the place of the box's store: the boxes take turns, and what store_read<1>
        // leaves pending has to be the other one's.
        if (lane == 0)
            store_commit();
        return;
    }
    unsigned char *const box = staging + c / WIDTH % 2 * BOX_BYTES;
    if (lane == 0)
        store_read<1>();
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        uint4 o;
        if constexpr (DH) {
            const float *x = v + u * 4;
            o = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        } else {
            const float *x = v + u * 8;
            o = make_uint4(pack2<DT>(x[0] * unit, x[1] * unit), pack2<DT>(x[2] * unit, x[3] * unit),
                           pack2<DT>(x[4] * unit, x[5] * unit), pack2<DT>(x[6] * unit, x[7] * unit));
        }
        *reinterpret_cast<uint4 *>(box + lane * 128 + ((u ^ (lane & 7)) * 16)) = o;
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (DH && a.first)
            tma_store(&a.dh, col + c, row, box);
        else if (DH)
            tma_add(&a.dh, col + c, row, box);
        else
            tma_store(&a.dw, col + c, a.v0 + row, box);
        store_commit();
    }
}

// A warp's 32 rows x 128 columns of a product to memory from the only sums of it in tensor memory (`free`: the
// barrier that gives the accumulators back; 0: there were no products, the sums are 0), where they are `wanted` (rows
// of a tile behind the last one are not): piece by piece, so that the first one is on its way early.
template <int DT, bool DH>
__device__ __forceinline__ void store_short(const ProductArgs &a, bool ok, uint32_t from, uint32_t free, int row, int col,
                                            bool wanted, float unit, unsigned char *staging, int lane)
{
    constexpr int WIDTH = PRODUCT_WIDTH<DH>;
#pragma unroll
    for (int c = 0; c < HALF; c += WIDTH) {
        float v[WIDTH];
        if (free) {
#pragma unroll
            for (int i = 0; i < WIDTH; i += 16)
                tmem_load16(from + c + i, reinterpret_cast<uint32_t *>(v + i));
            tmem_wait();
        } else {
#pragma unroll
            for (int i = 0; i < WIDTH; ++i)
                v[i] = 0.0f;
        }
        if (!ok) {  // (a wait ran out)
#pragma unroll
            for (int i = 0; i < WIDTH; ++i)
                v[i] = __builtin_nanf("");
        }
        if (c + WIDTH == HALF && free) {
            tmem_before();
            __syncwarp();
            if (lane == 0)
                arrive_at(free);
        }
        if (wanted)
            store_columns<DT, DH>(a, v, row, col, c, unit, staging, lane);
    }
}
// The same from registers.
template <int DT, bool DH>
__device__ __forceinline__ void store_long(const ProductArgs &a, const float (&z)[HALF], int row, int col, float unit,
                                           unsigned char *staging, int lane)
{
#pragma unroll
    for (int c = 0; c < HALF; c += PRODUCT_WIDTH<DH>)
        store_columns<DT, DH>(a, z + c, row, col, c, unit, staging, lane);
}

// LONG: sums in chunks of CHUNK_PRODUCTS blocks of K, where there are many rows or more than SHORT_PRODUCTS blocks of
// them; else one run.  (Tiles of many rows
// take the same time either way, as long as the registers stay below 168: with a split of them between the warps, as for
// the tiles of logits, the warp that issues products is too slow, and 4096 x 2048 x 50257 bf16 takes 1010 us instead of
// 934.  dw of few rows, which is no more than a way to memory, takes 161 us instead of 147 at 128 x 4096 x 32768.  There one
// thread issues the products: when they are issued faster, dh's reads and dw's writes mix less, 16 x 4096 x 50257 268 -> 281.)
template <int DT, bool LONG>
__global__ void __launch_bounds__(MMA_THREADS, 1) linear_products_kernel(const __grid_constant__ ProductArgs a)
{
    extern __shared__ unsigned char raw[];
    __shared__ MmaBarriers b;
    unsigned char *const ring = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = cluster_rank();
    mma_begin(b, warp, lane);
    pdl_enter();
    const int taken = a.work.head->live;
    // packed rows, with those of g's second parts
    const int live = a.few && taken > 0 && two_parts(taken, a.work.few) ? a.work.few / 2 + taken : taken;
    const int h_rows = a.with_dh ? (live + TILE - 1) / TILE : 0;
    const int w_rows = a.with_dw ? (a.v_count + TILE - 1) / TILE : 0;
    const int h_each = h_rows * a.n_tiles, h_tiles = h_each * a.splits, tiles = h_tiles + w_rows * a.n_tiles;
    const int v_blocks = (a.v_count + BLOCK_K - 1) / BLOCK_K, r_blocks = (live + BLOCK_K - 1) / BLOCK_K;
    const int v_each = (v_blocks + a.splits - 1) / a.splits;
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

    // The i-th tile of this pair: dh's in turn, then dw's.  A pair whose turn at dh does not come as
    // often as the others' gets as many more of dw's.  What a tile takes, in eighths of the time of one
    // block of K in the tensor cores: dh's its blocks, or 22 each where few rows of tiles share what a
    // block loads of the weights, dw's its blocks, or the 11 that its way to memory takes.
    // Of few rows dh is no more than reading and dw no more than writing, of 32 KB a block and 128 KB a
    // tile; memory reads and writes at once at 6.8 TB/s and only writes at 4, so beyond what L2 holds every
    // other pair begins with dw (gradient 128 x 4096 x 32768 209 -> 203 us; 64 x 1024 x 32001 63 -> 67).
    const int rest = h_tiles % pairs, w_tiles = tiles - h_tiles;
    const int h_cost = a.few ? v_each : v_each * max(8, 22 / max(h_rows, 1)), w_cost = a.few ? 4 : 8 * max(r_blocks, 11);
    const int more = rest == 0 ? 0 : min((h_cost + w_cost / 2) / w_cost, w_tiles / (pairs - rest));
    const int h_mine = h_tiles / pairs + (pair < rest), w_more = pair < rest ? 0 : more;
    const int w_shared = w_tiles - more * (pairs - rest);
    const int w_mine = w_more + w_shared / pairs + (pair < w_shared % pairs);
    const bool w_first = a.few && pair % 2 != 0 && w_tiles > 800;
    auto tile_of = [&](int i) {
        if (i >= h_mine + w_mine)
            return -1;
        i -= w_first ? w_mine : 0;
        i += i < 0 ? h_mine + w_mine : 0;  // as if dh's came first
        if (i < h_mine)
            return i * pairs + pair;
        i -= h_mine;
        return h_tiles + (i < w_more ? i * (pairs - rest) + pair - rest : more * (pairs - rest) + (i - w_more) * pairs + pair);
    };
    auto job = [&](int t) {
        if (t < h_tiles) {
            const int split = t / h_each, k = split * v_each;
            const TileAt at = tile_at(t - split * h_each, h_rows, a.n_tiles);
            return TileJob{&a.g_h, &a.w_n, at.m * TILE, at.n * TILE, k * BLOCK_K, a.v0 + k * BLOCK_K,
                           max(0, min(v_each, v_blocks - k)), !a.few, false};
        }
        t -= h_tiles;
        const TileAt at = a.few ? TileAt{t / a.n_tiles, t % a.n_tiles} : tile_at(t, w_rows, a.n_tiles);
        return TileJob{&a.g_w, &a.h_n, at.m * TILE, at.n * TILE, 0, 0, r_blocks, a.few, false};
    };
    if (warp == 0 && lane == 0) {
        RingPos<> pos;
        for (int i = 0, t; (t = tile_of(i)) >= 0; ++i)
            if (!copy_tile(job(t), b, ring, pos, rank)) {
                drain_copies(b, pos, rank);
                break;
            }
    } else if (warp == 1 && rank == 0 && (LONG || lane == 0)) {
        const bool issues = LONG ? elect_one() : true;
        RingPos<> pos;
        AccPos acc;
        for (int i = 0, t; (t = tile_of(i)) >= 0; ++i) {
            const TileJob j = job(t);
            if (!multiply_tile<LONG>(j, b, ring, pos, acc, instruction_desc(DT == RED_BF16, j.a_along_k, j.b_along_k),
                                     LONG ? CHUNK_PRODUCTS : SHORT_PRODUCTS, issues)) {
                drain_products(b, issues);
                break;
            }
        }
    } else if (warp >= 4) {
        AccPos acc;
        const int group = warp % 4, half = (warp - 4) / 4;
        uint32_t empty[2] = {leader_addr(&b.acc_empty[0]), leader_addr(&b.acc_empty[1])};
        unsigned char *const staging = ring + STAGES * STAGE_BYTES + (warp - 4) * STAGING_BYTES;
        const float unit = a.work.head->unit;
        for (int i = 0, t; (t = tile_of(i)) >= 0; ++i) {
            const TileJob j = job(t);
            const int row = j.a_row + rank * HALF + group * 32, col = j.b_row + half * HALF;
            if constexpr (LONG) {
                float z[HALF];
                if (!take_sums(z, b, acc, j.blocks, CHUNK_PRODUCTS, (uint32_t)(group * 32) << 16, half, empty) ||
                    j.blocks == 0) {
                    // a wait ran out, or there are no products
#pragma unroll
                    for (int k = 0; k < HALF; ++k)
                        z[k] = j.blocks == 0 ? 0.0f : __builtin_nanf("");
                }
                if (t >= h_tiles)
                    store_long<DT, false>(a, z, row, col, unit, staging, lane);
                else if (row < live)
                    store_long<DT, true>(a, z, row + t / h_each * (int)a.work.padded, col, unit, staging, lane);
            } else {
                const bool ok = j.blocks == 0 || mbar_wait(&b.acc_full[acc.slot], acc.phase, &b.failed, 0);
                tmem_after();
                const uint32_t from = b.tmem + ((uint32_t)(group * 32) << 16) + acc.slot * TILE + half * HALF;
                const uint32_t free = j.blocks == 0 ? 0 : empty[acc.slot];
                if (t < h_tiles)
                    store_short<DT, true>(a, ok, from, free, row + t / h_each * (int)a.work.padded, col, row < live, unit,
                                          staging, lane);
                else
                    store_short<DT, false>(a, ok, from, free, row, col, true, unit, staging, lane);
                if (j.blocks != 0)
                    acc.next();
            }
        }
        if (lane == 0)
            store_done();
    }
    __syncwarp();
    mma_end(b, warp);
}

// The sums of the pieces, and of their splits, to the rows' gradients, rounded once:
// a thread per four elements, or (SHARES 8) one of each of eight warps, an eighth of the
// splits each.  Zeros where a row takes no part.
template <int DT, int SHARES>
__global__ void __launch_bounds__(256)
    linear_scatter_kernel(const LinearWork w, int64_t rows, int64_t dim, uint16_t *dhidden, int64_t ldd)
{
    pdl_enter();
    constexpr int WIDTH = 256 / SHARES;
    __shared__ float4 shares[SHARES][WIDTH];
    const float unit = w.head->unit;
    const int64_t quads = w.dim4 / 4, split = w.padded * w.dim4;
    const int share = threadIdx.x / WIDTH, place = threadIdx.x % WIDTH;
    for (int64_t i0 = (int64_t)blockIdx.x * WIDTH; i0 < rows * quads; i0 += (int64_t)gridDim.x * WIDTH) {
        const int64_t i = i0 + place;
        const bool here = i < rows * quads;
        const int64_t r = here ? i / quads : 0, d = here ? (i - r * quads) * 4 : 0;
        const int at = here ? w.pos[r] : -1;
        uint16_t *to = dhidden + r * ldd + d;
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (at >= 0) {
            const float *from = w.dhidden + (int64_t)at * w.dim4 + d;
#pragma unroll 4
            for (int s = share; s < w.splits; s += SHARES) {
                const float4 v = *reinterpret_cast<const float4 *>(from + s * split);
                x[0] += v.x, x[1] += v.y, x[2] += v.z, x[3] += v.w;
            }
            if (two_parts(w.head->live, w.few)) {
                from += w.few / 2 * w.dim4;
                for (int s = share; s < w.splits; s += SHARES) {
                    const float4 v = *reinterpret_cast<const float4 *>(from + s * split);
                    x[0] += v.x, x[1] += v.y, x[2] += v.z, x[3] += v.w;
                }
            }
        }
        if constexpr (SHARES > 1) {
            __syncthreads();  // (the last round's shares have been read)
            shares[share][place] = make_float4(x[0], x[1], x[2], x[3]);
            __syncthreads();
            if (share != 0)
                continue;
#pragma unroll
            for (int k = 1; k < SHARES; ++k) {
                const float4 v = shares[k][place];
                x[0] += v.x, x[1] += v.y, x[2] += v.z, x[3] += v.w;
            }
        }
        if (!here)
            continue;
        if (d + 4 <= dim) {
            *reinterpret_cast<uint2 *>(to) =
                make_uint2(pack2<DT>(x[0] * unit, x[1] * unit), pack2<DT>(x[2] * unit, x[3] * unit));
        } else {
            for (int k = 0; k < 4 && d + k < dim; ++k)
                to[k] = (uint16_t)pack2<DT>(x[k] * unit, 0.0f);
        }
    }
}

// ------------------------------------------------------------------ launches

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn()
{
    static std::atomic<void *> cached{nullptr};
    void *f = cached.load(std::memory_order_relaxed);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        cached.store(f, std::memory_order_relaxed);
    }
    return reinterpret_cast<EncodeFn>(f);
}

// A matrix of `outer` rows of `inner` elements, row stride ld elements, in boxes
// with the 128-byte swizzle; what lies outside reads as zero and is not written.
int matrix_map(CUtensorMap *map, int dtype, const void *base, int64_t inner, int64_t outer, int64_t ld, int box_inner,
               int box_outer)
{
    const EncodeFn encode = encode_fn();
    if (!encode)
        return fail(RED_ECUDA, "the driver has no cuTensorMapEncodeTiled");
    const cuuint64_t sizes[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * (dtype == RED_F32 ? 4 : 2)};
    const cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_outer}, step[2] = {1, 1};
    const CUtensorMapDataType type = dtype == RED_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == RED_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUresult e = encode(map, type, 2, const_cast<void *>(base), sizes, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return e == CUDA_SUCCESS ? RED_OK : fail(RED_ECUDA, "cuTensorMapEncodeTiled: error %d", (int)e);
}

#define RETURN_IF(call)            \
    do {                           \
        const int st_ = (call);    \
        if (st_ != RED_OK)         \
            return st_;            \
    } while (0)

constexpr int MAX_DEVICES = 64;

// Pairs of CTAs of a kernel that run at once on the current device.
template <class Args>
int resident_pairs(void (*kernel)(const Args), std::atomic<int> (&cache)[MAX_DEVICES], int *pairs)
{
    DeviceInfo di;
    RETURN_IF(device_info(&di));
    int v = cache[di.dev].load(std::memory_order_relaxed);
    if (v == 0) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MMA_SMEM);
        if (e != cudaSuccess)
            return cuda_fail(e, "cudaFuncSetAttribute");
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)di.sms / 2 * 2);
        cfg.blockDim = dim3(MMA_THREADS);
        cfg.dynamicSmemBytes = MMA_SMEM;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&v, kernel, &cfg);
        if (e != cudaSuccess)
            return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
        if (v < 1)
            return fail(RED_ECUDA, "no pair of CTAs fits this device");
        cache[di.dev].store(v, std::memory_order_relaxed);
    }
    *pairs = v;
    return RED_OK;
}

template <class Args>
int launch_pairs(void (*kernel)(const Args), std::atomic<int> (&cache)[MAX_DEVICES], int64_t tiles, cudaStream_t s,
                 const Args &a, const char *what)
{
    int pairs;
    RETURN_IF(resident_pairs(kernel, cache, &pairs));
    if (tiles < pairs)
        pairs = (int)tiles;
    RETURN_IF(cuda_fail(launch_pdl_smem(kernel, 2u * (unsigned)pairs, MMA_THREADS, MMA_SMEM, 2, s, a), what));
    count_launches(1);
    return RED_OK;
}

template <int DT, bool GRAD>
int launch_logits(int64_t tiles, cudaStream_t s, const LogitArgs &a)
{
    static std::atomic<int> cache[MAX_DEVICES];
    return launch_pairs(linear_logits_kernel<DT, GRAD>, cache, tiles, s, a, "linear_logits");
}
template <int DT, bool LONG>
int launch_products(int64_t tiles, cudaStream_t s, const ProductArgs &a)
{
    static std::atomic<int> cache[MAX_DEVICES];
    return launch_pairs(linear_products_kernel<DT, LONG>, cache, tiles, s, a, "linear_products");
}
template <int DT>
int launch_products(int64_t tiles, cudaStream_t s, const ProductArgs &a)
{
    // dw alone of up to 1024 rows, too, is bound by its way to memory (719 x 6976 x 3827 94 us, 115 by the other kernel; 1000 x
    // 1024 x 50257 152, 153; with dh 126 and 211, 125 and 209 by the other)
    const int64_t blocks = up(a.v_count, BLOCK_K) / BLOCK_K;  // of dh
    const bool is_short = a.few ? (blocks + a.splits - 1) / a.splits <= SHORT_PRODUCTS : !a.with_dh && a.work.padded <= 1024;
    return is_short ? launch_products<DT, false>(tiles, s, a) : launch_products<DT, true>(tiles, s, a);
}

template <int DT, bool GRAD, int ROWS>
int launch_few_rows(const LinearArgs &l, FewArgs &a, unsigned *grid, cudaStream_t s)
{
    static std::atomic<bool> ready[MAX_DEVICES];
    DeviceInfo di;
    RETURN_IF(device_info(&di));
    auto *const kernel = linear_few_kernel<DT, GRAD, ROWS>;
    if (!ready[di.dev].load(std::memory_order_relaxed)) {
        RETURN_IF(cuda_fail(
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Few<ROWS, GRAD>::SMEM),
            "cudaFuncSetAttribute"));
        ready[di.dev].store(true, std::memory_order_relaxed);
    }
    // equal shares of whole tiles; a share of less than 16 columns is not worth a CTA
    const int most = di.sms < FEW_MAX_CTAS ? di.sms : FEW_MAX_CTAS;
    const int share = a.vocab / most < 16 ? 16 : (a.vocab + most - 1) / most;
    a.tiles = (share + HALF - 1) / HALF;
    a.height = (share + a.tiles - 1) / a.tiles;
    *grid = (unsigned)((a.vocab + a.tiles * a.height - 1) / (a.tiles * a.height));
    RETURN_IF(matrix_map(&a.w, l.dtype, l.weight, l.dim, l.vocab, l.ldw, BLOCK_K, a.height));
    RETURN_IF(cuda_fail(launch_pdl_smem(kernel, *grid, FEW_THREADS, Few<ROWS, GRAD>::SMEM, 1, s, a), "linear_few"));
    count_launches(1);
    return RED_OK;
}
// `grid`: the CTAs that it took, one slot of the statistics each.
template <bool GRAD>
int launch_few(const LinearArgs &a, const LinearWork &w, unsigned *grid, cudaStream_t s)
{
    FewArgs f;
    if (GRAD)
        RETURN_IF(matrix_map(&f.h, a.dtype, w.hidden, a.dim, w.padded, w.ld, BLOCK_K, w.few));
    else
        RETURN_IF(matrix_map(&f.h, a.dtype, a.hidden, a.dim, a.rows, a.ldh, BLOCK_K, w.few));
    f.targets = a.target;
    f.rows = (int)a.rows;
    f.work = w;
    f.vocab = (int)a.vocab;
    f.k_blocks = (int)(up(a.dim, BLOCK_K) / BLOCK_K);
    f.s2 = (float)(a.scale * 1.4426950408889634);
#define FEW_OF(rows) \
    (a.dtype == RED_BF16 ? launch_few_rows<RED_BF16, GRAD, rows>(a, f, grid, s)          \
                           : launch_few_rows<RED_F16, GRAD, rows>(a, f, grid, s))
    return w.few == 16 ? FEW_OF(16) : w.few == 32 ? FEW_OF(32) : w.few == 64 ? FEW_OF(64) : FEW_OF(128);
#undef FEW_OF
}

unsigned warp_rows_grid(int64_t rows) { return (unsigned)((rows + 7) / 8 < 65536 ? (rows + 7) / 8 : 65536); }

template <bool GRAD>
int pack_rows(const LinearArgs &a, const LinearWork &w, const float *lse, const float *dlogp, const float *dlse,
              cudaStream_t s)
{
    const ScanArgs scan = {a, lse, dlogp, dlse, w};
    if (a.rows <= GATHER_ROWS) {
        count_launches(1);
        return cuda_fail(launch_pdl(a.rows <= 1024 ? linear_gather_kernel<GRAD, 4> : linear_gather_kernel<GRAD, 16>,
                                    dim3((unsigned)(w.padded / 8)), dim3(256), s, scan),
                         "linear_gather");
    }
    RETURN_IF(cuda_fail(launch_pdl(linear_scan_kernel<GRAD>, dim3(1), dim3(SCAN_NT), s, scan), "linear_scan"));
    RETURN_IF(cuda_fail(launch_pdl(linear_pack_kernel<GRAD>, dim3(warp_rows_grid(w.padded)), dim3(256), s, scan),
                        "linear_pack"));
    count_launches(2);
    return RED_OK;
}

}  // namespace

LinearWork linear_work(void *base, int64_t rows, int64_t dim, int64_t vocab, bool grad)
{
    LinearWork w = {};
    if (rows == 0)
        return w;
    unsigned char *const p = static_cast<unsigned char *>(base);
    int64_t at = 0;
    auto take = [&](auto *&field, int64_t bytes) {
        field = reinterpret_cast<std::remove_reference_t<decltype(field)>>(p + at);
        at += up(bytes, 256);
    };
    w.padded = up(rows, TILE);
    w.ld = up(dim, 8);
    w.dim4 = up(dim, 4);
    w.few = rows > FEW_ROWS ? 0 : rows > 64 ? 128 : rows > 32 ? 64 : rows > 16 ? 32 : 16;
    // Of up to 16 rows there is room for g in two parts (two_parts()): 1 x 2048 x 65536 184.4 -> 186.8 us, 16 x 4096 x 50257
    // 268.4 -> 269.9.  Always so up to 32 rows 32 x 2048 x 65536 takes 190.5 instead of 187.5, up to 64 rows 64 x 1024 x 32001
    // 62.5 instead of 57.6: of that many rows the error is 1.2 to 1.4 times the results' rounding without.
    if (grad && rows <= 16)
        w.few = rows <= 8 ? 16 : 32;
    w.slots = w.few ? FEW_MAX_CTAS : up(vocab, TILE) / HALF;
    take(w.head, sizeof(LinearHead));
    take(w.pos, rows * 4);
    take(w.idx, rows * 4);
    take(w.target, rows * 4);
    uint16_t *h, *g;
    take(h, w.padded * w.ld * 2);
    w.hidden = h;
    if (!grad) {
        take(w.part, rows * w.slots * 8);
    } else {
        // A piece's gradient by the logits takes 256 MiB, and 4096 columns where rows are more than 32768: narrower
        // pieces pass over the sums of dh too often (262144 x 512 x 32768 bf16: 20.6 ms, 29.8 in pieces of 2048 columns;
        // 524288 x 256 x 32768 34.9, 91.7 in pieces of 1024).  That goes up to 8 GiB; beyond 2^20 rows
        // pieces are narrower all the same, down to a tile's 256 columns.  Pieces are of equal width,
        // which may be half as much again, or one tile more: a narrow last one leaves CTAs without work.
        const int64_t most = ((int64_t)1 << 32) / w.padded;
        int64_t cols = ((int64_t)1 << 27) / w.padded;
        cols = cols < 4096 ? (most < 4096 ? most : 4096) : cols;
        cols = cols < TILE ? TILE : cols / TILE * TILE;
        const int64_t pieces = w.few ? 1 : (2 * vocab + cols) / (2 * cols);
        w.piece_cols = up((vocab + (pieces > 1 ? pieces : 1) - 1) / (pieces > 1 ? pieces : 1), TILE);
        take(w.at_target, rows * 4);
        take(w.by_p, rows * 4);
        take(w.lse2, rows * 4);
        take(g, (w.few ? w.few : w.padded) * w.piece_cols * 2);
        w.piece = g;
        // dh of few rows is few tiles that are long: shares of the vocabulary fill the pairs of CTAs
        // (64 x 1024 x 32001: four tiles of 501 blocks of K, products 191 us, in 18 shares 46)
        const int64_t tiles = w.padded / TILE * (up(dim, TILE) / TILE), blocks = w.piece_cols / BLOCK_K;
        int64_t splits = w.piece_cols < up(vocab, TILE) ? 1 : 72 / tiles;
        splits = splits < blocks / 8 ? splits : blocks / 8;
        w.splits = splits < 1 ? 1 : (int)splits;
        take(w.dhidden, w.splits * w.padded * w.dim4 * 4);
    }
    w.bytes = at;
    return w;
}

int launch_linear_logprob(const LinearArgs &a, float *logp, float *lse, void *work, cudaStream_t s)
{
    const LinearWork w = linear_work(work, a.rows, a.dim, a.vocab, false);
    if (!w.few)
        RETURN_IF(pack_rows<false>(a, w, nullptr, nullptr, nullptr, s));
    const float s2 = (float)(a.scale * 1.4426950408889634);
    int64_t slots = w.slots;
    if (w.few) {
        unsigned grid;
        RETURN_IF(launch_few<false>(a, w, &grid, s));
        slots = grid;
    } else {
        LogitArgs l;
        RETURN_IF(matrix_map(&l.h, a.dtype, w.hidden, a.dim, w.padded, w.ld, BLOCK_K, HALF));
        RETURN_IF(matrix_map(&l.w, a.dtype, a.weight, a.dim, a.vocab, a.ldw, BLOCK_K, HALF));
        l.g = l.w;
        l.work = w;
        l.v0 = 0;
        l.n_tiles = (int)(up(a.vocab, TILE) / TILE);
        l.vocab = (int)a.vocab;
        l.k_blocks = (int)(up(a.dim, BLOCK_K) / BLOCK_K);
        l.chunk = even_chunk(l.k_blocks);
        l.s2 = s2;
        const int64_t tiles = w.padded / TILE * l.n_tiles;
        RETURN_IF((a.dtype == RED_BF16 ? launch_logits<RED_BF16, false>(tiles, s, l)
                                       : launch_logits<RED_F16, false>(tiles, s, l)));
    }
    const bool wide = a.rows <= 2048;
    RETURN_IF(cuda_fail(launch_pdl(wide ? linear_join_kernel<256> : linear_join_kernel<32>,
                                   dim3(wide ? (unsigned)a.rows : warp_rows_grid(a.rows)), dim3(256), s, a, w, slots, s2,
                                   logp, lse),
                        "linear_join"));
    count_launches(1);
    return RED_OK;
}

int launch_linear_logprob_grad(const LinearArgs &a, const float *lse, const float *dlogp, const float *dlse,
                               void *dhidden, int64_t ldd, void *dweight, int64_t lddw, void *work, cudaStream_t s)
{
    const LinearWork w = linear_work(work, a.rows, a.dim, a.vocab, true);
    RETURN_IF(pack_rows<true>(a, w, lse, dlogp, dlse, s));
    LogitArgs l;
    ProductArgs p;
    RETURN_IF(matrix_map(&l.h, a.dtype, w.hidden, a.dim, w.padded, w.ld, BLOCK_K, HALF));
    RETURN_IF(matrix_map(&l.w, a.dtype, a.weight, a.dim, a.vocab, a.ldw, BLOCK_K, HALF));
    if (w.few) {
        RETURN_IF(matrix_map(&p.g_h, a.dtype, w.piece, w.few, a.vocab, w.few, 64, BLOCK_K));
        RETURN_IF(matrix_map(&p.g_w, a.dtype, w.piece, w.few, a.vocab, w.few, BLOCK_K, HALF));
    } else {
        RETURN_IF(matrix_map(&l.g, a.dtype, w.piece, w.piece_cols, w.padded, w.piece_cols, 64, 32));
        RETURN_IF(matrix_map(&p.g_h, a.dtype, w.piece, w.piece_cols, w.padded, w.piece_cols, BLOCK_K, HALF));
        RETURN_IF(matrix_map(&p.g_w, a.dtype, w.piece, w.piece_cols, w.padded, w.piece_cols, 64, BLOCK_K));
    }
    p.few = w.few != 0;
    RETURN_IF(matrix_map(&p.w_n, a.dtype, a.weight, a.dim, a.vocab, a.ldw, 64, BLOCK_K));
    RETURN_IF(matrix_map(&p.h_n, a.dtype, w.hidden, a.dim, w.padded, w.ld, 64, BLOCK_K));
    RETURN_IF(matrix_map(&p.dh, RED_F32, w.dhidden, a.dim, w.padded * w.splits, w.dim4, 32, 32));
    if (dweight)
        RETURN_IF(matrix_map(&p.dw, a.dtype, dweight, a.dim, a.vocab, lddw, 64, 32));
    else
        p.dw = p.w_n;
    l.work = p.work = w;
    l.vocab = (int)a.vocab;
    l.k_blocks = (int)(up(a.dim, BLOCK_K) / BLOCK_K);
    l.chunk = CHUNK_GRAD;
    l.s2 = (float)(a.scale * 1.4426950408889634);
    p.n_tiles = (int)(up(a.dim, TILE) / TILE);
    p.splits = w.splits;
    p.with_dh = dhidden != nullptr;
    p.with_dw = dweight != nullptr;
    p.dweight = static_cast<uint16_t *>(dweight);
    p.lddw = lddw;
    p.dim = (int)a.dim;
    p.vocab = (int)a.vocab;
    for (int64_t v0 = 0; v0 < a.vocab; v0 += w.piece_cols) {
        const int64_t count = a.vocab - v0 < w.piece_cols ? a.vocab - v0 : w.piece_cols;
        l.v0 = p.v0 = (int)v0;
        l.n_tiles = (int)(up(count, TILE) / TILE);
        p.v_count = (int)count;
        p.first = v0 == 0;
        const int64_t m_tiles = w.padded / TILE;
        const int64_t tiles = (p.with_dh ? m_tiles * w.splits : 0) * p.n_tiles + (int64_t)(p.with_dw ? l.n_tiles : 0) * p.n_tiles;
        unsigned grid;
        if (w.few)
            RETURN_IF(launch_few<true>(a, w, &grid, s));
        else
            RETURN_IF((a.dtype == RED_BF16 ? launch_logits<RED_BF16, true>(m_tiles * l.n_tiles, s, l)
                                           : launch_logits<RED_F16, true>(m_tiles * l.n_tiles, s, l)));
        RETURN_IF((a.dtype == RED_BF16 ? launch_products<RED_BF16>(tiles, s, p) : launch_products<RED_F16>(tiles, s, p)));
    }
    if (dhidden) {
        // A CTA's places: 256, or 32 in eight shares.  The whole gradient, us, without / with shares: 18 splits (64 x 1024 x
        // 32001) 61 / 58, 9 (300 x 1024 x 8192) 38 / 39, 4 (128 x 4096 x 32768) 206 / 211.
        const bool shares = w.splits >= 16;
        auto *const kernel = a.dtype == RED_BF16
                                 ? (shares ? linear_scatter_kernel<RED_BF16, 8> : linear_scatter_kernel<RED_BF16, 1>)
                                 : (shares ? linear_scatter_kernel<RED_F16, 8> : linear_scatter_kernel<RED_F16, 1>);
        const unsigned grid = warp_rows_grid(a.rows * w.dim4 / 4 / (shares ? 4 : 32) + 1);
        RETURN_IF(cuda_fail(launch_pdl(kernel, dim3(grid), dim3(256), s, w, a.rows, a.dim, static_cast<uint16_t *>(dhidden), ldd),
                            "linear_scatter"));
        count_launches(1);
    }
    return RED_OK;
}

}  // namespace red
