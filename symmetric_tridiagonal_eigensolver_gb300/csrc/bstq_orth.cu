// Orthogonalised update: Newton-Schulz products that bring the singular
// values of a matrix near one.  Kernels and the entry point.
//
// A step is X <- a X + (b A + c A^2) X with A = X X^T, X being p x q with
// p <= q (a tall matrix is transposed on the way in and out).  It runs as
// three products on the fp16 tensor cores with sums in 32 bits:
//
//   E = A - theta I        X X^T, upper tiles only, mirrored as they are stored
//   B = (b + 2 c theta) E + c E^2        E E, upper tiles only
//   X <- (a + b theta + c theta^2) X + B X
//
// which is the same polynomial for any theta (expanded about A = theta I).
// What theta does is place the roundings.  With theta = 0 the term B X has
// nothing in the directions of small singular values, whose share comes
// exactly from a X; roundings there would be amplified by a = 3.4445 in each
// step to come.  With theta = 1 B X has little in the directions whose singular
// values have come near one, where |b A + c A^2| is 2.7 at theta = 0.  So
// theta is 0 but for the last two steps, 1/2 and 1 there: relative error of the
// bf16 result on 512 x 512 normal and low-rank matrices 1.8e-3 and 2.3e-3
// against 2.2e-3 and 1.8e-3 with 0 throughout and 1.9e-3 and 1.7e-2 with 1 in the last four
// (1.7e-3 is the output's own rounding).
//
// Numbers: X is kept as two fp16 terms (22 bits) times 2^14, E as 2^12 E, B as
// 2^10 B, which leaves room for singular values up to 2.  The factors of the
// products are the leading terms alone for bf16 (11 bits, eight times finer
// than the result) and both terms, in three products, for float and half.
// X_0 is G times a power of two (bf16 and half exactly, float to 22 bits); 1 / |G|
// enters as a factor of sums in the first step, so that no rounding by it is amplified.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/bstq.h"
#include "bstq_common.h"
#include "bstq_orth_plan.h"
#include "bstq_pack.cuh"
#include "bstq_tensor.cuh"

namespace bstq {
namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }

constexpr float kXs = 16384.0f;  // X is stored times this,
constexpr float kEs = 4096.0f;   // E times this
constexpr float kBs = 1024.0f;   // and B times this

// ---------------------------------------------------------------------------
// Norm and first iterate
// ---------------------------------------------------------------------------
constexpr int kNormThreads = 256;
constexpr int kNormMaxParts = 256;  // blocks per matrix in the norm's first pass

// A sum of squares, sum * 4^back.  It is taken as it is where that ends between 2^-90
// and 2^118, else once more with every value times 2^100 or 2^-100: for a whole matrix
// in the small kernel, for what one block adds up here, of which up to 256 come
// together below 2^128.  No element is in another unit than its neighbours, so G times
// a power of two goes through the same roundings.
struct Sq {
    float sum;
    int back;  // -100, 0 or 100
};
__device__ __forceinline__ int back_of(float plain)  // 100 for a NaN too
{
    return plain <= 0x1p-90f ? -100 : (plain < 0x1p118f ? 0 : 100);
}
__device__ __forceinline__ float factor_of(int back) { return back > 0 ? 0x1p-100f : 0x1p100f; }
// The sum in units of 4^back, back being at least its own or the sum zero.
__device__ __forceinline__ float in_units(Sq s, int back)
{
    if (s.back == back)
        return s.sum;
    return back - s.back == 100 ? s.sum * 0x1p-100f * 0x1p-100f : 0.0f;
}

__device__ __forceinline__ float block_sum(float v, float *sm)
{
    for (int d = 16; d; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        sm[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int i = 0; i < kNormThreads / 32; ++i)
        t += sm[i];
    return t;
}

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }

struct Scale {
    int e;       // X_0 is stored as G * 2^e
    float unit;  // X_0 = unit * stored
};
// Norm = 2^k f with 1 <= f < 2, in units of 2^back.
__device__ __forceinline__ Scale scale_of(Sq s)
{
    if (!(s.sum < INFINITY))
        return Scale{0, nanf("")};
    if (s.sum == 0.0f)
        return Scale{0, 0.0f};
    const float norm = sqrtf(s.sum);
    const int k = ilogbf(norm);
    // stored norm: norm 2^back 2^e = f 2^14
    return Scale{14 - k - s.back, 1.0f / ldexpf(norm, 14 - k)};
}

// Eight neighbouring values, of which `count` are there; the others are zero.
__device__ __forceinline__ void read8(const float *g, int count, bool vector, float (&v)[8])
{
    if (vector && count >= 8) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(g)), b = __ldg(reinterpret_cast<const float4 *>(g) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = k < count ? g[k] : 0.0f;
}
template <typename T>
__device__ __forceinline__ void read8(const T *g, int count, bool vector, float (&v)[8])
{
    if (vector && count >= 8) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(g));
        const T *t = reinterpret_cast<const T *>(&w);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = to_f(t[k]);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = k < count ? to_f(g[k]) : 0.0f;
}

// Sums of squares: pieces of eight consecutive values (of the matrix, row by
// row), in one order whatever the row stride; four to a thread in flight.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    norm_kernel(const T *G, long long sb, long long sr, long long m, long long n, int parts, bool vector, Sq *part,
                int *status)
{
    __shared__ float sm[kNormThreads / 32];
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *status = 0;
    const T *g = G + (long long)blockIdx.y * sb;
    const long long all = m * n, pieces = (all + 7) / 8, step = (long long)parts * kNormThreads;
    auto each = [&](auto add) {
        for (long long i = (long long)blockIdx.x * kNormThreads + threadIdx.x; i < pieces; i += 4 * step) {
            float v[4][8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const long long at = 8 * (i + u * step);
                const int count = at >= all ? 0 : (all - at < 8 ? (int)(all - at) : 8);
                if (sr == n) {
                    read8(g + at, count, vector, v[u]);
                } else {
                    long long row = at / n, col = at - row * n;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        v[u][k] = k < count ? to_f(g[row * sr + col]) : 0.0f;
                        if (++col == n)
                            col = 0, ++row;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    add(v[u][k]);
        }
    };
    float plain = 0.0f;
    each([&](float v) { plain = fmaf(v, v, plain); });
    plain = block_sum(plain, sm);
    const int back = back_of(plain);
    if (back != 0) {
        const float f = factor_of(back);
        plain = 0.0f;
        each([&](float v) { plain = fmaf(v * f, v * f, plain); });
        plain = block_sum(plain, sm);
    }
    if (threadIdx.x == 0)
        part[(long long)blockIdx.y * parts + blockIdx.x] = Sq{plain, back};
}

__device__ __forceinline__ void two_terms(float v, __half &hi, __half &lo)
{
    hi = __float2half_rn(v);
    lo = __float2half_rn(v - __half2float(hi));
}

// X_0 in two planes of p x ld (p <= q <= ld), rows padded with zeros, in pieces of
// eight columns; a tall G goes through a 64 x 32 tile in shared memory.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    start_kernel(const T *G, long long sb, long long sr, bool tall, int parts, bool vector, const Sq *part, __half *X, int p,
                 int q, int ld, float *unit)
{
    __shared__ float sm[kNormThreads / 32];
    __shared__ float tile[64][33];
    const long long b = blockIdx.z;
    Sq s{0.0f, -100};
    if ((int)threadIdx.x < parts)
        s = part[b * parts + threadIdx.x];
    const bool held = s.sum != 0.0f;
    const int back = __syncthreads_or(held && s.back > 0) ? 100 : (__syncthreads_or(held && s.back == 0) ? 0 : -100);
    const Scale sc = scale_of(Sq{block_sum(in_units(s, back), sm), back});
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        unit[b] = sc.unit;
    // 2^e in two factors, each in range
    const Pk<2> f0 = pk_all<2>(power_of_two(sc.e / 2)), f1 = pk_all<2>(power_of_two(sc.e - sc.e / 2));
    const T *g = G + b * sb;
    __half *hi = X + b * 2 * (long long)p * ld, *lo = hi + (long long)p * ld;
    auto place = [&](int r, int c, const float (&v)[8]) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            two_terms_open(mul_(mul_(Pk<2>::make(v[2 * k], v[2 * k + 1]), f0), f1), h[k], l[k]);
        *reinterpret_cast<uint4 *>(hi + (long long)r * ld + c) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(lo + (long long)r * ld + c) = make_uint4(l[0], l[1], l[2], l[3]);
    };
    // blocks of 64 columns and 32 rows
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, px = threadIdx.x & 7, py = threadIdx.x >> 3;
    for (int r0 = blockIdx.y * 32; r0 < p; r0 += gridDim.y * 32) {
        for (int c0 = blockIdx.x * 64; c0 < ld; c0 += gridDim.x * 64) {
            float v[8];
            const int r = r0 + py, c = c0 + 8 * px;
            if (tall) {
                __syncthreads();
                float in[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int col = c0 + ty + 8 * i;
                    in[i] = col < q && r0 + tx < p ? to_f(g[(long long)col * sr + r0 + tx]) : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    tile[ty + 8 * i][tx] = in[i];
                __syncthreads();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = tile[8 * px + k][py];
            } else if (r < p) {
                read8(g + (long long)r * sr + c, q - c, vector, v);
            }
            if (r < p && c < ld)
                place(r, c, v);
        }
    }
}

// ---------------------------------------------------------------------------
// The products
// ---------------------------------------------------------------------------
enum { EPI_GRAM = 0, EPI_SQUARE = 1, EPI_UPDATE = 2, EPI_LAST = 3 };

struct ProductArgs {
    int p, q;         // E and B are p x p, X is p x q
    int ldx, lds;     // row lengths of X's and of E's and B's planes
    int k;            // length of the sums
    int tiles_m, tiles_n, tiles;  // tiles per matrix
    long long batch;
    const __half *in;   // EPI_SQUARE: E; EPI_UPDATE, EPI_LAST: X
    const float *unit;  // X = unit * stored, per matrix; NULL: 1 / kXs
    float c0, c1;       // GRAM: theta; SQUARE: b + 2 c theta, c; else a + b theta + c theta^2
    void *last;         // EPI_LAST: the caller's result
    long long last_b, last_r;
    int flip, vector;   // write it transposed; its rows' pieces of eight start on 16 bytes
    int *status;
    long long wait;     // cycles after which a wait gives up
};

constexpr int kBM = 128, kBK = 64;
constexpr int kOutBytes = 4096;  // of each warp that takes sums out: two pieces of 32 x 32 fp16 values

// CTAS == 2: a pair of blocks works on a tile of 256 rows, each with its 128 rows
// of the left factor and half of the columns of the right one: 32 KB for a block of
// K that the tensor cores take 512 cycles for, against 48 KB of a 128 x 256 tile
// (2 x 4096 x 4096 bf16 at burst clocks: 2.12 ms without pairs, 1.82 with).
template <int BN, int PLANES, int CTAS>
struct Shape {
    static constexpr int kA = kBM * kBK * 2, kB = BN / CTAS * kBK * 2;
    static constexpr int kStage = PLANES * (kA + kB);
    static constexpr int kStages = (192 * 1024) / kStage;
    static constexpr int kSmem = 1024 + kStages * kStage + 8 * kOutBytes;
    // Tensor memory: two accumulators in turn.  Every product added to a sum
    // there costs it a rounding towards zero, so with two planes (float, half)
    // a sum is taken out and added up in registers each kChunk blocks of K,
    // and the products of a leading and a second term have sums of their own,
    // one per tile in turn (1531 x 777 float: 7.9e-6 off with one running sum,
    // 6.6e-6 with the second apart, 0.8e-6 with both; a 32-bit library product:
    // 3.1e-6).
    static constexpr int kChunk = PLANES == 2 ? 4 : 1 << 30;
    static constexpr int kColumns = PLANES * 2 * BN;
};

constexpr int kEpiWarps = 8;
constexpr int kProductThreads = 32 * (4 + kEpiWarps);

// The tile'th tile of a matrix: all of them row by row for an update, those
// that reach the diagonal or lie above it for E and B.
template <int BN, int CTAS, bool UPPER>
__device__ __forceinline__ void tile_at(const ProductArgs &a, int t, int &i, int &j)
{
    if (!UPPER) {
        j = t / a.tiles_m;
        i = t - j * a.tiles_m;
        return;
    }
    i = 0;
    for (;;) {
        const int first = i * CTAS * kBM / BN, count = a.tiles_n - first;
        if (t < count) {
            j = first + t;
            return;
        }
        t -= count;
        ++i;
    }
}

__device__ __forceinline__ void store_last(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_last(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_last(__half *p, float v) { *p = __float2half_rn(v); }

template <typename T>
struct alignas(16) Row8 {
    T v[8];
};

// What a tile's element was before: 32 values of one row of X or E, as loaded.
template <int PLANES, int EPI>
struct Before {
    static constexpr bool X = EPI == EPI_UPDATE || EPI == EPI_LAST;
    static constexpr int kPlanes = EPI == EPI_GRAM ? 0 : (X ? 2 : PLANES);
    uint4 w[kPlanes ? kPlanes : 1][4];
    __device__ __forceinline__ void load(const ProductArgs &a, long long b, int row, int col)
    {
        const int ld = X ? a.ldx : a.lds;
        const long long plane = (long long)a.p * ld;
        const __half *in = a.in + b * 2 * plane + (long long)row * ld + col;
#pragma unroll
        for (int pl = 0; pl < kPlanes; ++pl)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                w[pl][g] = row < a.p && col + 8 * g < ld ? __ldcg(reinterpret_cast<const uint4 *>(in + pl * plane + 8 * g))
                                                          : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ Pk<2> get(int k) const  // values 2 k and 2 k + 1
    {
        const uint4 &h = w[0][k >> 2];
        const uint32_t hw = (k & 3) == 0 ? h.x : ((k & 3) == 1 ? h.y : ((k & 3) == 2 ? h.z : h.w));
        if constexpr (kPlanes == 2) {
            const uint4 &l = w[1][k >> 2];
            const uint32_t lw = (k & 3) == 0 ? l.x : ((k & 3) == 1 ? l.y : ((k & 3) == 2 ? l.z : l.w));
            return add_(from_half2(hw), from_half2(lw));
        }
        return from_half2(hw);
    }
};

// 32 x 32 values of a warp (lane: row), as fp16 pieces through shared memory to
// a plane: 64-byte rows whose 16-byte parts are permuted as TMA's 64-byte swizzle
// has them.
__device__ __forceinline__ void piece_rows(char *piece, const uint32_t (&w)[16], int lane)
{
#pragma unroll
    for (int g = 0; g < 4; ++g)
        *reinterpret_cast<uint4 *>(piece + lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
}
// the same transposed: lane is the column
__device__ __forceinline__ void piece_columns(char *piece, const uint32_t (&w)[16], int lane)
{
#pragma unroll
    for (int k = 0; k < 32; ++k)
        *reinterpret_cast<uint16_t *>(piece + k * 64 + (((lane >> 3) ^ ((k >> 1) & 3)) << 4) + (lane & 7) * 2) =
            (uint16_t)(k & 1 ? w[k >> 1] >> 16 : w[k >> 1]);
}
__device__ __forceinline__ void piece_store(const CUtensorMap *map, const char *piece, int col, int row, int plane, int lane)
{
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
        tma_store(map, smem_u32(piece), col, row, plane);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}
// every piece stored so far may be overwritten
__device__ __forceinline__ void pieces_free(int lane)
{
    if (lane == 0)
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}

// 32 columns of a warp's 32 rows, from the sums to where they go.  `mirror`: to
// the transposed place too.
template <int PLANES, int EPI, typename T>
__device__ __forceinline__ void epilogue32(const ProductArgs &a, const CUtensorMap &out, char *pieces, long long b, int row,
                                           int col, Pk<2> (&v)[16], const Before<PLANES, EPI> &before, float unit,
                                           bool mirror, int lane)
{
    if constexpr (EPI == EPI_GRAM) {
        const Pk<2> f = pk_all<2>(unit * unit * kEs);
        const int pair = (row - col) >> 1;
        const Pk<2> off = row & 1 ? Pk<2>::make(0.0f, -kEs * a.c0) : Pk<2>::make(-kEs * a.c0, 0.0f);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            v[k] = mul_(v[k], f);
            if (k == pair)
                v[k] = add_(v[k], off);
        }
    } else {
        const float x0 = EPI == EPI_SQUARE ? a.c0 * (kBs / kEs) : (EPI == EPI_UPDATE ? unit * kXs : unit) * a.c0;
        const float s0 = EPI == EPI_SQUARE ? a.c1 * (kBs / kEs / kEs)
                                           : (EPI == EPI_UPDATE ? unit * kXs : unit) * (1.0f / kBs);
#pragma unroll
        for (int k = 0; k < 16; ++k)
            v[k] = fma_(pk_all<2>(x0), before.get(k), mul_(pk_all<2>(s0), v[k]));
    }
    if constexpr (EPI == EPI_LAST) {
        if (row >= a.p)
            return;
        T *const to = (T *)a.last + b * a.last_b;
        if (a.flip) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
                if (col + k < a.q)
                    store_last(to + (long long)(col + k) * a.last_r + row, v[k >> 1].get(k & 1));
            return;
        }
        T *const at = to + (long long)row * a.last_r + col;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            Row8<T> y;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                store_last(&y.v[k], v[4 * g + k / 2].get(k & 1));
            if (a.vector && col + 8 * g + 8 <= a.q) {
                *reinterpret_cast<Row8<T> *>(at + 8 * g) = y;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (col + 8 * g + k < a.q)
                        at[8 * g + k] = y.v[k];
            }
        }
    } else {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
            two_terms_open(v[k], hi[k], lo[k]);
        constexpr int N = EPI == EPI_UPDATE ? 2 : PLANES;  // X keeps both terms
        const int row0 = row - lane, z = (int)(2 * b);
        pieces_free(lane);
        piece_rows(pieces, hi, lane);
        if (N == 2)
            piece_rows(pieces + 2048, lo, lane);
        piece_store(&out, pieces, col, row0, z, lane);
        if (N == 2)
            piece_store(&out, pieces + 2048, col, row0, z + 1, lane);
        if (EPI != EPI_UPDATE && mirror) {
            if (N == 2)
                pieces_free(lane);
            piece_columns(N == 2 ? pieces : pieces + 2048, hi, lane);
            if (N == 2)
                piece_columns(pieces + 2048, lo, lane);
            piece_store(&out, N == 2 ? pieces : pieces + 2048, row0, col, z, lane);
            if (N == 2)
                piece_store(&out, pieces + 2048, row0, col, z + 1, lane);
        }
    }
}

// Persistent: one block per SM (or pair of blocks on two) walks tiles of 128 x BN
// (256 x BN).  Warp 0 loads (TMA,
// 128-byte swizzle, kStages deep), warp 1 issues the products, eight warps
// take the sums out of tensor memory while the next tile's products run, and
// store by TMA, in place and mirrored (with 2-byte stores of the mirrored half
// X X^T of 777 x 1531 float took 22 us, by TMA 15.6, and E E 18.4 and 12.1).
//
// What bounds it: a block takes 64 bytes a cycle from L2, in which a pair's tile of
// 256 x 256 just keeps the tensor cores busy; 2 x 4096 x 4096 bf16 runs at 1.3
// PFLOP/s in a stream of passes, where the power limit holds (77 % of the measured
// sustained rate), and at 1.5 at burst clocks.  With fewer tiles than SMs one tile's way
// along K is the time, and below 1024 rows the way in and out: some 9 us a product
// of 512 x 512, of which 1.3 are the first copy's latency, 3.8 the products, 1.4 the
// sums' way out.  Sharing a tile's K among several blocks, in a cluster or through
// memory, cost more there than it gained (125 -> 147 and 159 us).
template <int BN, int PLANES, int CTAS, bool B_MN, int EPI, typename T>
__global__ void __launch_bounds__(kProductThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap left, const __grid_constant__ CUtensorMap right,
                   const __grid_constant__ CUtensorMap out, const __grid_constant__ ProductArgs a)
{
    using S = Shape<BN, PLANES, CTAS>;
    constexpr bool UPPER = EPI == EPI_GRAM || EPI == EPI_SQUARE;
    extern __shared__ char raw[];
    __shared__ uint64_t bars[2 * S::kStages + 5];
    __shared__ uint32_t tmem_slot;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S::kStages + s); };
    auto tfull = [&](int s) { return bar0 + 8u * (2 * S::kStages + s); };
    auto tempty = [&](int s) { return bar0 + 8u * (2 * S::kStages + 2 + s); };
    const uint32_t issued = bar0 + 8u * (2 * S::kStages + 4);  // all products are done
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(tfull(s), 1);
            mbar_init(tempty(s), CTAS * kEpiWarps);
        }
        mbar_init(issued, 1);
        mbar_init_fence();
    }
    if (warp == 2)
        tmem_alloc<CTAS>(smem_u32(&tmem_slot), S::kColumns);
    tc_before();
    __syncthreads();
    if (CTAS == 2) {  // the other block's barriers are there
        cluster_arrive();
        cluster_wait();
    }
    tc_after();
    const int rank = CTAS == 2 ? (int)cluster_rank() : 0;
    const long long tile0 = blockIdx.x / CTAS, tiles_by = gridDim.x / CTAS;
    // the next product's blocks may come; what the last one wrote is read from here on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = tmem_slot;
    const long long total = a.batch * a.tiles;
    const int steps = (a.k + kBK - 1) / kBK;

    if (warp == 0) {
        if (elect_one()) {
            int s = 0;
            uint32_t phase = 0;
            for (long long t = tile0; t < total; t += tiles_by) {
                const long long b = t / a.tiles;
                int i, j;
                tile_at<BN, CTAS, UPPER>(a, (int)(t - b * a.tiles), i, j);
                bool ok = true;
                for (int k = 0; k < steps && ok; ++k) {
                    if (!mbar_wait(empty(s), phase ^ 1, a.wait)) {
                        *a.status = 1;
                        ok = false;
                        break;
                    }
                    const uint32_t at = base + s * S::kStage;
                    // the leader's barrier counts both blocks' bytes
                    const uint32_t bar = CTAS == 2 ? at_rank(full(s), 0) : full(s);
                    if (rank == 0)
                        mbar_expect(full(s), CTAS * S::kStage);
                    auto load = [&](uint32_t to, const CUtensorMap *map, int x, int y, int z) {
                        if (CTAS == 2)
                            tma_load_pair(to, map, bar, x, y, z);
                        else
                            tma_load(to, map, bar, x, y, z);
                    };
                    const int left_row = (i * CTAS + rank) * kBM, right_col = j * BN + rank * (BN / CTAS);
#pragma unroll
                    for (int pl = 0; pl < PLANES; ++pl) {
                        const int z = (int)(2 * b) + pl;
#pragma unroll
                        for (int h = 0; h < kBM / 64; ++h)
                            load(at + pl * S::kA + h * 8192, &left, k * kBK, left_row + h * 64, z);
                        const uint32_t bt = at + PLANES * S::kA + pl * S::kB;
#pragma unroll
                        for (int h = 0; h < BN / CTAS / 64; ++h)
                            if (B_MN)
                                load(bt + h * 8192, &right, right_col + h * 64, k * kBK, z);
                            else
                                load(bt + h * 8192, &right, k * kBK, right_col + h * 64, z);
                    }
                    if (++s == S::kStages)
                        s = 0, phase ^= 1;
                }
                if (!ok)
                    break;
            }
            // no copy is still on its way in when the block ends, whoever gave up
            if (rank == 0)
                for (int k = 0; k < S::kStages; ++k)
                    mbar_wait(full(k), k < s ? phase : phase ^ 1);
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = mma_desc(CTAS * kBM, BN, B_MN);
            int s = 0, acc = 0, side = 0;
            uint32_t phase = 0, aphase = 0;
            bool ok = true;
            for (long long t = tile0; t < total && ok; t += tiles_by) {
                const uint32_t cross = tmem + 2 * BN + side * BN;
                side ^= 1;
                for (int k = 0; k < steps; ++k) {
                    const bool first = k % S::kChunk == 0;
                    if (first) {
                        if (!(ok = mbar_wait(tempty(acc), aphase ^ 1, a.wait)))
                            break;
                        tc_after();
                    }
                    const uint32_t d = tmem + acc * BN;
                    if (!(ok = mbar_wait(full(s), phase, a.wait)))
                        break;
                    tc_after();
                    const uint32_t at = base + s * S::kStage, bt = at + PLANES * S::kA;
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        uint64_t da[PLANES], db[PLANES];
#pragma unroll
                        for (int pl = 0; pl < PLANES; ++pl) {
                            da[pl] = desc_k(at + pl * S::kA + kk * 32);
                            db[pl] = B_MN ? desc_mn(bt + pl * S::kB + kk * 2048, 8192) : desc_k(bt + pl * S::kB + kk * 32);
                        }
                        tc_mma<CTAS>(d, da[0], db[0], idesc, !first || kk > 0);
                        if (PLANES == 2) {
                            tc_mma<CTAS>(cross, da[0], db[PLANES - 1], idesc, k + kk > 0);
                            tc_mma<CTAS>(cross, da[PLANES - 1], db[0], idesc, true);
                        }
                    }
                    tc_commit<CTAS>(empty(s));
                    if (++s == S::kStages)
                        s = 0, phase ^= 1;
                    if (k == steps - 1 || (k + 1) % S::kChunk == 0) {
                        tc_commit<CTAS>(tfull(acc));
                        if (++acc == 2)
                            acc = 0, aphase ^= 1;
                    }
                }
            }
            if (!ok)
                *a.status = 1;
            tc_commit<CTAS>(issued);  // nor any product
            mbar_wait(issued, 0);
        } else if (rank == 1 && elect_one()) {
            mbar_wait(issued, 0);  // nor an arrival from the other block
        }
    } else if (warp >= 4) {
        // warp w reads lanes 32 (w mod 4) and up, and one half of the columns
        const int w = warp - 4, quarter = w & 3, half = w >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + half * (BN / 2);
        char *const pieces = raw + (base - smem_u32(raw)) + S::kStages * S::kStage + w * kOutBytes;
        constexpr int C = BN / 64;  // groups of 32 columns
        auto leave = [&](int acc) {  // the sums are out: to the block that issues the products
            if (CTAS == 2)
                mbar_arrive_far(at_rank(tempty(acc), 0));
            else
                mbar_arrive(tempty(acc));
        };
        int acc = 0, side = 0;
        uint32_t aphase = 0;
        // Where a wait ran out, in this product or in one before, the result is no
        // number; a warp that gave up goes on without waiting or handing on.
        const bool wrong = EPI == EPI_LAST && __ldcg(a.status) != 0;
        bool ok = true;
        auto sums_there = [&] {
            if (ok && !__all_sync(0xffffffffu, mbar_wait(tfull(acc), aphase, a.wait))) {
                *(volatile int *)a.status = 1;
                ok = false;
            }
            tc_after();
        };
        for (long long t = tile0; t < total; t += tiles_by) {
            const long long b = t / a.tiles;
            int i, j;
            tile_at<BN, CTAS, UPPER>(a, (int)(t - b * a.tiles), i, j);
            i = i * CTAS + rank;  // this block's 128 rows
            const float stored = a.unit ? __ldcg(a.unit + b) : 1.0f / kXs;
            const int row = i * kBM + quarter * 32 + lane, col = j * BN + half * (BN / 2);
            // of the symmetric ones a square of 128 above the diagonal goes to both
            // places, one on it to its own, one below is another tile's
            auto wanted = [&](int c) { return !UPPER || (col + 32 * c) / kBM >= i; };
            auto mirror = [&](int c) { return UPPER && (col + 32 * c) / kBM > i; };
            Before<PLANES, EPI> before;
            before.load(a, b, row, col);
            if (PLANES == 1) {
                sums_there();
                const float unit = wrong || !ok ? nanf("") : stored;
#pragma unroll 1
                for (int c = 0; c < C; ++c) {
                    float f[32];
                    tmem_load32(lanes + acc * BN + 32 * c, f);
                    tmem_load_wait();
                    Pk<2> v[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        v[k] = Pk<2>::make(f[2 * k], f[2 * k + 1]);
                    const Before<PLANES, EPI> now = before;
                    if (c + 1 < C)
                        before.load(a, b, row, col + 32 * (c + 1));
                    if (wanted(c))
                        epilogue32<PLANES, EPI, T>(a, out, pieces, b, row, col + 32 * c, v, now, unit, mirror(c), lane);
                }
                tc_before();
                __syncwarp();
                if (ok && lane == 0)
                    leave(acc);
                if (++acc == 2)
                    acc = 0, aphase ^= 1;
            } else {
                Pk<2> sum[C][16];
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        sum[c][k] = pk_all<2>(0.0f);
                for (int k = 0; k < steps; k += S::kChunk) {
                    sums_there();
                    const bool last = k + S::kChunk >= steps;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        float f[32];
                        tmem_load32(lanes + acc * BN + c * 32, f);
                        tmem_load_wait();
#pragma unroll
                        for (int n = 0; n < 16; ++n)
                            sum[c][n] = add_(sum[c][n], Pk<2>::make(f[2 * n], f[2 * n + 1]));
                        if (last) {
                            tmem_load32(lanes + 2 * BN + side * BN + c * 32, f);
                            tmem_load_wait();
#pragma unroll
                            for (int n = 0; n < 16; ++n)
                                sum[c][n] = add_(sum[c][n], Pk<2>::make(f[2 * n], f[2 * n + 1]));
                        }
                    }
                    tc_before();
                    __syncwarp();
                    if (ok && lane == 0)
                        leave(acc);
                    if (++acc == 2)
                        acc = 0, aphase ^= 1;
                }
                side ^= 1;
                const float unit = wrong || !ok ? nanf("") : stored;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    if (c)
                        before.load(a, b, row, col + 32 * c);
                    if (wanted(c))
                        epilogue32<PLANES, EPI, T>(a, out, pieces, b, row, col + 32 * c, sum[c], before, unit, mirror(c),
                                                   lane);
                }
            }
        }
        if (lane == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    if (CTAS == 2) {  // no block leaves while the other uses its memory or barriers
        cluster_arrive();
        cluster_wait();
    }
    if (warp == 2)
        tmem_free<CTAS>(tmem, S::kColumns);
}

}  // namespace
}  // namespace bstq

#include "bstq_orth_small.cuh"

namespace bstq {
namespace {

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr float kCoefs[3] = {3.4445f, -4.7750f, 2.0315f};
constexpr int kMaxSteps = 32;

bool takes(bstq_dtype d) { return d == BSTQ_F32 || d == BSTQ_BF16 || d == BSTQ_F16; }
// Planes are counted in 32 bits and blocks of a grid's z axis in 16.
bool sizes_ok(int64_t batch, int64_t m, int64_t n)
{
    return batch >= 0 && batch <= 65535 && m >= 0 && n >= 0 && m <= (1 << 20) && n <= (1 << 20) &&
           (double)batch * m * n <= (double)(1LL << 38);
}
size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

// The widest cluster of the small kernel that the device places; asked once for each.
// Clusters of 16 are beyond what every device or part of one has room for: there the
// sizes that need them go in tiles.  Without a device, sizes are those of one that has.
int widest_cluster()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return kWidestCluster;
    }
    int widest = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (widest)
        return widest;
    auto *fn = small_kernel<__nv_bfloat16, 1, 256, true, false>;  // no other takes more shared memory
    typedef SmallShape<1, 256, true, false> S;
    static_assert(S::kSmem >= SmallShape<2, 256, true, false>::kSmem, "");
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    widest = 1;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) == cudaSuccess &&
        cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess)
        for (int blocks = kWidestCluster; blocks > 1 && widest == 1; blocks /= 2) {
            int clusters = 0;
            at.val.clusterDim.x = (unsigned)blocks;
            cfg.gridDim = dim3((unsigned)blocks);
            if (cudaOccupancyMaxActiveClusters(&clusters, fn, &cfg) == cudaSuccess && clusters > 0)
                widest = blocks;
        }
    cudaGetLastError();  // a size that the device has not is no error of the caller's
    if (dev < 64)
        known[dev].store(widest, std::memory_order_relaxed);
    return widest;
}

struct OrthPlan {
    int p, q, ldx, lds, parts;
    size_t part, unit, x0, x1, e, b, total;  // byte offsets in the workspace; its first 256 bytes hold the status
};
OrthPlan plan_of(int64_t batch, int64_t m, int64_t n)
{
    OrthPlan s{};
    s.p = (int)(m < n ? m : n), s.q = (int)(m < n ? n : m);
    s.ldx = (s.q + 7) & ~7, s.lds = (s.p + 7) & ~7;
    const int64_t want = (m * n + 8191) / 8192;  // four pieces of eight to a thread
    s.parts = (int)(want < 1 ? 1 : (want > kNormMaxParts ? kNormMaxParts : want));
    if (is_small(m, n, widest_cluster())) {
        s.total = 256;
        return s;
    }
    const size_t x = round256(4 * size_t(batch) * s.p * s.ldx), e = round256(4 * size_t(batch) * s.p * s.lds);
    s.part = 256;
    s.unit = s.part + round256(sizeof(Sq) * s.parts * batch);
    s.x0 = s.unit + round256(4 * size_t(batch));
    s.x1 = s.x0 + x;
    s.e = s.x1 + x;
    s.b = s.e + e;
    s.total = s.b + e;
    return s;
}

// Map of 2 * batch planes of rows x ld fp16 values, read in boxes of 64 x 64
// (128-byte swizzle) or written in boxes of 32 x 32 (64-byte swizzle); what a box
// has beyond rows x cols reads as zero and is not written.
cudaError_t planes_map(CUtensorMap *map, const void *at, int rows, int cols, int ld, int64_t batch, unsigned side)
{
    const EncodeFn fn = encode_fn();
    if (!fn)
        return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)(2 * batch)};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * rows};
    const cuuint32_t box[3] = {side, side, 1}, unit[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(at), dims, strides, box, unit,
              CU_TENSOR_MAP_INTERLEAVE_NONE, side == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

int tiles_of(int p, int cols, int bm, int bn, bool upper)
{
    const int tm = (p + bm - 1) / bm, tn = (cols + bn - 1) / bn;
    if (!upper)
        return tm * tn;
    int t = 0;
    for (int i = 0; i < tm; ++i)
        t += tn - i * bm / bn;
    return t;
}

template <int BN, int PLANES, int CTAS, int EPI, typename T>
cudaError_t launch_tiles(const CUtensorMap &l, const CUtensorMap &r, const CUtensorMap &o, ProductArgs a, int sms,
                         cudaStream_t s)
{
    constexpr bool upper = EPI == EPI_GRAM || EPI == EPI_SQUARE;
    const int cols = upper ? a.p : a.q;
    a.tiles_m = (a.p + CTAS * kBM - 1) / (CTAS * kBM);
    a.tiles_n = (cols + BN - 1) / BN;
    a.tiles = tiles_of(a.p, cols, CTAS * kBM, BN, upper);
    auto *fn = product_kernel<BN, PLANES, CTAS, !upper, EPI, T>;
    constexpr int smem = Shape<BN, PLANES, CTAS>::kSmem;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(CTAS);
    cfg.blockDim = dim3(kProductThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CTAS;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    // asked once for each device: the blocks, or pairs (not every SM has a
    // partner), that run at once
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    int room = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (room == 0) {
        if ((err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
            return err;
        room = sms;
        if (CTAS == 2) {
            cfg.numAttrs = 1;
            if ((err = cudaOccupancyMaxActiveClusters(&room, fn, &cfg)) != cudaSuccess)
                return err;
            room = room > 0 ? room : 1;
        }
        if (dev < 64)
            known[dev].store(room, std::memory_order_relaxed);
    }
    const long long total = a.batch * a.tiles;
    cfg.gridDim = dim3((unsigned)((total < room ? total : room) * CTAS));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, l, r, o, a);
}

// The tile by the rounds that the SMs need: a tile costs its columns and some 32
// more (the way in and out), a round as much as a tile; in pairs a tile's rows are
// twice as many and its time some 0.8 of two single ones'.  Measured with one
// product's tile forced, a pass of five steps: B X of 2 x 4096 x 4096 bf16 1.89 ms in
// pairs of 256 columns, 2.00 of 128, 1.97 and 2.10 in single blocks; of 2048 x 8192
// 636, 611, 652 and 632 us; X X^T and E E of 1531 x 777 float 243 in pairs of 128,
// 249 and 210 in single blocks of 128 and 64.  The rule's choice is the best of them or
// within 2 %.  Every width adds a sum's terms in the same order, so a matrix's result
// does not depend on its batch.
template <int PLANES, int EPI, typename T>
cudaError_t launch_product(const CUtensorMap &l, const CUtensorMap &r, const CUtensorMap &o, const ProductArgs &a, int sms,
                           cudaStream_t s)
{
    constexpr bool upper = EPI == EPI_GRAM || EPI == EPI_SQUARE;
    auto cost = [&](int ctas, int bn) {
        const long long total = a.batch * tiles_of(a.p, upper ? a.p : a.q, ctas * kBM, bn, upper);
        const long long at_once = sms / ctas;
        return (total + at_once - 1) / at_once * (double)(bn * (ctas == 2 ? 0.8 : 1.0) + 32.0);
    };
    constexpr int wide = PLANES == 1 ? 256 : 128;
    int bn = 64, ctas = 1;
    double best = cost(1, 64);
    auto consider = [&](int c, int n) {
        const double d = cost(c, n);
        if (d <= best)
            best = d, ctas = c, bn = n;
    };
    consider(1, 128);
    if (PLANES == 1)
        consider(1, 256);
    consider(2, 128);
    consider(2, wide);
    if (ctas == 2)
        return bn == 128 ? launch_tiles<128, PLANES, 2, EPI, T>(l, r, o, a, sms, s)
                         : launch_tiles<wide, PLANES, 2, EPI, T>(l, r, o, a, sms, s);
    if (bn == 64)
        return launch_tiles<64, PLANES, 1, EPI, T>(l, r, o, a, sms, s);
    if (bn == 128)
        return launch_tiles<128, PLANES, 1, EPI, T>(l, r, o, a, sms, s);
    return launch_tiles<wide, PLANES, 1, EPI, T>(l, r, o, a, sms, s);
}

template <typename T>
struct PlanesOf {
    static constexpr int value = 2;
};
template <>
struct PlanesOf<__nv_bfloat16> {
    static constexpr int value = 1;
};

template <typename T, int PL, int QC, bool CL, bool STACK>
cudaError_t launch_small(const SmallArgs &a, long long groups, int ranks, cudaStream_t s)
{
    auto *fn = small_kernel<T, PL, QC, CL, STACK>;
    constexpr int smem = SmallShape<PL, QC, CL, STACK>::kSmem;
    static std::atomic<bool> known[64];  // set once for each device
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    if (dev >= 64 || !known[dev].load(std::memory_order_relaxed)) {
        if ((err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
            (CL && (err = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess))
            return err;
        if (dev < 64)
            known[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(groups * ranks));
    cfg.blockDim = dim3(SmallShape<PL, QC, CL, STACK>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ranks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = CL ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

template <typename T, int PL>
cudaError_t run_small(const SmallArgs &a, cudaStream_t s)
{
    const long long stacked = 128 >> a.log_rows, groups = (a.batch + stacked - 1) / stacked;
    if (a.q <= 64)
        return launch_small<T, PL, 64, false, true>(a, groups, 1, s);
    if (a.q <= 128)
        return a.p <= 64 ? launch_small<T, PL, 128, false, true>(a, groups, 1, s)
                         : launch_small<T, PL, 128, false, false>(a, groups, 1, s);
    if (a.q <= 256)
        return launch_small<T, PL, 256, false, false>(a, groups, 1, s);
    return launch_small<T, PL, 256, true, false>(a, groups, cluster_of(a.q), s);
}

template <typename T>
cudaError_t orthogonalize(int64_t batch, int64_t m, int64_t n, const T *G, T *X, const int64_t *st, int steps,
                          const float *coefs, char *work, int sms, cudaStream_t s)
{
    constexpr int PLANES = PlanesOf<T>::value;
    cudaError_t err;
    if (is_small(m, n, widest_cluster())) {
        SmallArgs a{};
        a.G = G, a.X = X, a.gb = st[0], a.gr = st[1], a.xb = st[2], a.xr = st[3], a.batch = batch;
        a.tall = m > n, a.p = (int)(a.tall ? n : m), a.q = (int)(a.tall ? m : n), a.steps = steps;
        a.log_rows = a.p > 64 ? 7 : (a.p > 32 ? 6 : (a.p > 16 ? 5 : 4));
        a.status = (int *)work, a.wait = wait_limit();
        const int lead = 16 / (int)sizeof(T);
        a.vector = !misaligned_to(G, 16) && st[1] % lead == 0 && st[0] % lead == 0;
        a.vector_out = !a.tall && !misaligned_to(X, 16) && st[3] % lead == 0 && st[2] % lead == 0;
        for (int i = 0; i < 3 * steps; ++i)
            a.coefs[i] = coefs[i];
        // few rows average few roundings: two planes there whatever the type
        return PLANES == 2 || a.p <= 32 ? run_small<T, 2>(a, s) : run_small<T, PLANES>(a, s);
    }
    const OrthPlan pl = plan_of(batch, m, n);
    Sq *part = (Sq *)(work + pl.part);
    float *unit = (float *)(work + pl.unit);
    __half *x[2] = {(__half *)(work + pl.x0), (__half *)(work + pl.x1)};
    __half *e = (__half *)(work + pl.e), *bb = (__half *)(work + pl.b);
    CUtensorMap mx[2], me, mb, ox[2], oe, ob;
    for (int k = 0; k < 2; ++k)
        if ((err = planes_map(&mx[k], x[k], pl.p, pl.q, pl.ldx, batch, 64)) != cudaSuccess ||
            (err = planes_map(&ox[k], x[k], pl.p, pl.q, pl.ldx, batch, 32)) != cudaSuccess)
            return err;
    if ((err = planes_map(&me, e, pl.p, pl.p, pl.lds, batch, 64)) != cudaSuccess ||
        (err = planes_map(&oe, e, pl.p, pl.p, pl.lds, batch, 32)) != cudaSuccess ||
        (err = planes_map(&mb, bb, pl.p, pl.p, pl.lds, batch, 64)) != cudaSuccess ||
        (err = planes_map(&ob, bb, pl.p, pl.p, pl.lds, batch, 32)) != cudaSuccess)
        return err;
    const int lead = 16 / (int)sizeof(T);
    const bool vector = !misaligned_to(G, 16) && st[0] % lead == 0 && st[1] % lead == 0;
    norm_kernel<T><<<dim3(pl.parts, (unsigned)batch), kNormThreads, 0, s>>>(
        G, st[0], st[1], m, n, pl.parts, !misaligned_to(G, 16) && st[0] % lead == 0, part, (int *)work);
    const unsigned gx = (pl.ldx + 63) / 64, gy = (pl.p + 31) / 32;
    start_kernel<T><<<dim3(gx < 64 ? gx : 64, gy < 64 ? gy : 64, (unsigned)batch), kNormThreads, 0, s>>>(
        G, st[0], st[1], m > n, pl.parts, vector, part, x[0], pl.p, pl.q, pl.ldx, unit);
    if ((err = cudaGetLastError()) != cudaSuccess)
        return err;
    for (int k = 0; k < steps; ++k) {
        const float ca = coefs[3 * k], cb = coefs[3 * k + 1], cc = coefs[3 * k + 2];
        const float theta = k == steps - 1 ? 1.0f : (k == steps - 2 ? 0.5f : 0.0f);
        ProductArgs a{};
        a.p = pl.p, a.q = pl.q, a.ldx = pl.ldx, a.lds = pl.lds, a.batch = batch, a.status = (int *)work;
        a.wait = wait_limit();
        a.unit = k == 0 ? unit : nullptr;
        const int from = k & 1, to = from ^ 1;
        a.k = pl.q, a.c0 = theta;
        if ((err = launch_product<PLANES, EPI_GRAM, float>(mx[from], mx[from], oe, a, sms, s)) != cudaSuccess)
            return err;
        a.k = pl.p, a.in = e, a.c0 = cb + 2.0f * cc * theta, a.c1 = cc;
        if ((err = launch_product<PLANES, EPI_SQUARE, float>(me, me, ob, a, sms, s)) != cudaSuccess)
            return err;
        a.in = x[from], a.c0 = ca + theta * (cb + theta * cc);
        a.last = X, a.last_b = st[2], a.last_r = st[3], a.flip = m > n;
        a.vector = !misaligned_to(X, 16) && st[2] % lead == 0 && st[3] % lead == 0;
        err = k + 1 < steps ? launch_product<PLANES, EPI_UPDATE, float>(mb, mx[from], ox[to], a, sms, s)
                            : launch_product<PLANES, EPI_LAST, T>(mb, mx[from], ox[to], a, sms, s);
        if (err != cudaSuccess)
            return err;
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace bstq

using namespace bstq;

extern "C" size_t bstq_orthogonalize_work_size(bstq_dtype dtype, int64_t batch, int64_t m, int64_t n)
{
    if (!takes(dtype) || !sizes_ok(batch, m, n))
        return 0;
    return plan_of(batch, m, n).total;
}

extern "C" int bstq_orthogonalize(bstq_dtype dtype, int64_t batch, int64_t m, int64_t n, const void *G, void *X,
                                  const int64_t *strides, int steps, const float *coefs, void *work, void *stream)
{
    if (!takes(dtype))
        return -1;
    if (batch < 0 || batch > 65535)
        return -2;
    if (m < 0 || m > (1 << 20))
        return -3;
    if (!sizes_ok(batch, m, n))
        return -4;
    if (batch == 0 || m == 0 || n == 0)
        return 0;
    const size_t e = dtype == BSTQ_F32 ? 4 : 2;
    if (!G || misaligned_to(G, e))
        return -5;
    if (!X || misaligned_to(X, e))
        return -6;
    const int64_t dense[4] = {m * n, n, m * n, n};
    const int64_t *st = strides ? strides : dense;
    for (int i = 0; i < 4; ++i)
        if (st[i] < 0 || st[i] > (1LL << 42))
            return -7;
    if (!rows_apart(n, m, st[3], batch, st[2]))
        return -7;
    if (steps < 1 || steps > kMaxSteps)
        return -8;
    float c[3 * kMaxSteps];
    for (int i = 0; i < 3 * steps; ++i) {
        c[i] = coefs ? coefs[i] : kCoefs[i % 3];
        if (!(fabsf(c[i]) <= (i % 3 ? 32.0f : 16.0f)))
            return -9;
    }
    if (!work || misaligned_to(work, 256))
        return -10;
    DevInfo di;
    if (!dev_info(di))
        return BSTQ_ERR_NODEVICE;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t err;
    if (dtype == BSTQ_F32)
        err = orthogonalize<float>(batch, m, n, (const float *)G, (float *)X, st, steps, c, (char *)work, di.sms, s);
    else if (dtype == BSTQ_BF16)
        err = orthogonalize<__nv_bfloat16>(batch, m, n, (const __nv_bfloat16 *)G, (__nv_bfloat16 *)X, st, steps, c,
                                           (char *)work, di.sms, s);
    else
        err = orthogonalize<__half>(batch, m, n, (const __half *)G, (__half *)X, st, steps, c, (char *)work, di.sms, s);
    return err == cudaSuccess ? 0 : cuda_fail(err, "orthogonalised update");
}
