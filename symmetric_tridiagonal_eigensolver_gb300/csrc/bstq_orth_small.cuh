// Orthogonalised update of small matrices, min(m, n) <= 128, in one launch: the
// iterates stay in shared and tensor memory from the first to the last step.
//
// A block (or a cluster of up to 16, each with up to 256 columns) holds 128
// rows: one matrix, or several of at most 64, 32 or 16 rows one below the other.
// Stacked matrices meet in X X^T only, whose blocks off the diagonal are set to
// zero, so E and B are block diagonal and E E and B X act on each matrix alone.
// With at most 64 rows a matrix (STACK) a row of E keeps the 64 columns of its own
// half: E E then has 64 terms, and B X is one product with the two halves of X side
// by side, of which each row reads its own (1024 x 64 x 64 float: 74 -> 67 us, three
// blocks to an SM instead of two).
// (A zero times another matrix's NaN would not be zero: a matrix that is not
// finite is left out, as zeros, and its result set to NaN at the end.)
//
// X's two fp16 planes lie in 128-byte swizzled rows, which serve as K-contiguous
// factor of X X^T and as N-contiguous factor of B X.  In a cluster a block owns
// 128 / C rows of E: it reads the C blocks' partial sums of X X^T, adds them up in
// order of rank and writes its rows into every block.
//
// What bounds it: the chain of three products a step, each with a pass through
// registers after it.  A step of 64 x 64 float takes some 8000 cycles: 1000, 1900 and
// 1500 in the three products (their latency in it; E E has since lost half its
// terms) and 1200 to 1300 in each pass.  1024 x 64 x 64 float: 66 us, 512 blocks,
// three to an SM; its 33.5 MB and 16 GFLOP would take 8.  32 x 128 x 1024 bf16: 70 us
// in clusters of four, 10.5 a step, half of it the exchange of E (two cluster
// barriers and 64 KB a block); 32 x 128 x 256, without the exchange, 36 us.
#pragma once

namespace bstq {
namespace {

struct SmallArgs {
    const void *G;
    void *X;
    long long gb, gr, xb, xr;  // element strides of batch and row
    long long batch;
    int p, q, tall, log_rows, steps;
    int vector, vector_out;  // whether pieces of eight of G and of X start on 16 bytes
    float coefs[3 * 32];
    int *status;
    long long wait;  // cycles after which a wait gives up
};

template <int PL, int QC, bool CL, bool STACK>
struct SmallShape {
    static constexpr int kX = QC / 64 * 16384;           // one plane of X
    static constexpr int kPlane = STACK ? 16384 : 32768;  // one of E: 128 rows of 64 or 128 columns
    static constexpr int kE = PL * kPlane;
    // a cluster's partial sums: beside E where there is room, else in its place
    static constexpr bool kBeside = CL && PL == 1;
    static constexpr int kSmem = 1024 + 2 * kX + kE + (kBeside ? 65536 : 0);
    // One sum for all three products of two planes: those of a leading and a second
    // term go first, while the sum is small and its rounding with it.
    static constexpr int kCols = STACK ? 2 * QC : (QC > 128 ? QC : 128);
    // Passes through registers take most of a step: sixteen warps where a block
    // has an SM to itself (32 x 128 x 1024 bf16: 79 us with eight, 73 with sixteen),
    // eight where two or three blocks share it.
    static constexpr int kThreads = STACK ? 256 : 512;
    // Blocks to an SM that the registers are kept for; none asked for otherwise (asking
    // for one made 32 x 128 x 1024 bf16 71 us instead of 67).
    static constexpr int kBlocks = STACK ? (QC == 64 ? 3 : 2) : 0;
};

struct SmallShared {
    float warp[16], part[16][8];  // [rank][matrix]
    Sq sum[8];
    Scale scale[8];
    int bad[8], stop;
    uint64_t done, drained;
    uint32_t tmem;
};

__device__ __forceinline__ float4 far_load(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ void far_store(uint32_t addr, uint4 v)
{
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ void far_store(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Byte offset of (row, col) in planes of 128 rows: blocks of 64 columns, rows of
// 128 bytes, the 16-byte pieces of a row permuted by the row's last three bits.
__device__ __forceinline__ uint32_t swizzled(int row, int col)
{
    return (uint32_t)((col >> 6) * 16384 + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2);
}

// Eight values in a plane and (PL == 2) their second terms in the other.
template <int PL>
__device__ __forceinline__ void store8(char *at, int other, const Pk<2> (&v)[4], float &top)
{
    uint4 hi, lo;
    two_terms(v[0], hi.x, lo.x, top);
    two_terms(v[1], hi.y, lo.y, top);
    two_terms(v[2], hi.z, lo.z, top);
    two_terms(v[3], hi.w, lo.w, top);
    *reinterpret_cast<uint4 *>(at) = hi;
    if (PL == 2)
        *reinterpret_cast<uint4 *>(at + other) = lo;
}
template <int PL>
__device__ __forceinline__ void load8(const char *at, int other, Pk<2> (&v)[4])
{
    const uint4 hi = *reinterpret_cast<const uint4 *>(at);
    v[0] = from_half2(hi.x), v[1] = from_half2(hi.y), v[2] = from_half2(hi.z), v[3] = from_half2(hi.w);
    if (PL == 2) {
        const uint4 lo = *reinterpret_cast<const uint4 *>(at + other);
        v[0] = add_(v[0], from_half2(lo.x)), v[1] = add_(v[1], from_half2(lo.y));
        v[2] = add_(v[2], from_half2(lo.z)), v[3] = add_(v[3], from_half2(lo.w));
    }
}

template <typename T, int PL, int QC, bool CL, bool STACK>
__global__ void __launch_bounds__(SmallShape<PL, QC, CL, STACK>::kThreads, SmallShape<PL, QC, CL, STACK>::kBlocks)
    small_kernel(const __grid_constant__ SmallArgs a)
{
    using S = SmallShape<PL, QC, CL, STACK>;
    extern __shared__ char raw[];
    __shared__ SmallShared sm;
    char *const xs = (char *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    char *const es = xs + 2 * S::kX;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ranks = CL ? (int)cluster_size() : 1, rank = CL ? (int)cluster_rank() : 0;
    const int rows = 1 << a.log_rows, stacked = 128 >> a.log_rows;
    const long long b0 = (long long)(blockIdx.x / ranks) * stacked;
    const int c0 = rank * QC;
    const int width = a.q - c0 < QC ? (a.q > c0 ? a.q - c0 : 0) : QC;
    const T *const G = (const T *)a.G;

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&sm.done), 1);
        mbar_init(smem_u32(&sm.drained), 1);
        mbar_init_fence();
    }
    if (threadIdx.x < 8)
        sm.bad[threadIdx.x] = 0;
    if (threadIdx.x == 0)
        sm.stop = 0;
    if (warp == 0)
        tmem_alloc(smem_u32(&sm.tmem), S::kCols);
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *(volatile int *)a.status = 0;
    if (CL) {  // every block of the cluster runs before another writes into it
        cluster_arrive();
        cluster_wait();
    }

    // G comes in pieces of eight values that are neighbours in memory (along a row
    // of X, or for a tall G along a column); a warp has eight or sixteen rows, which
    // are one matrix's, and kFlight pieces to a lane in flight.
    constexpr int kRows = 128 / (S::kThreads / 32);  // of a warp
    const int r0 = warp * kRows, mine = r0 >> a.log_rows, i0 = r0 & (rows - 1);
    const bool here = b0 + mine < a.batch;
    const T *const mat = G + (b0 + mine) * a.gb;
    const int span = (width + 63) & ~63;  // columns that a product reads
    const int per_row = span >> 3, pieces = span * kRows / 256;
    constexpr int kFlight = 4;
    auto where = [&](int n, int &r, int &c) {  // the n'th piece of a lane: row within the warp's, column
        const int id = lane + 32 * n;
        if (a.tall) {
            r = id % (kRows / 8) * 8;
            c = id / (kRows / 8);
        } else {
            r = id / per_row;
            c = (id - r * per_row) * 8;
        }
    };
    auto fetch = [&](int n, float (&v)[8]) {
        int r, c;
        where(n, r, c);
        const int i = i0 + r;
        const int count = !here || n >= pieces ? 0 : (a.tall ? (c < width ? a.p - i : 0) : (i < a.p ? width - c : 0));
        read8(a.tall ? mat + (c0 + c) * a.gr + i : mat + i * a.gr + c0 + c, count, a.vector, v);
    };

    // ---- the norms: sums of squares, once more in another unit where a matrix's whole
    // sum shows that 32 bits do not hold it
    int back = 0;  // of this warp's matrix
    for (bool again = false;; again = true) {
        const float f = back ? factor_of(back) : 1.0f;
        float sum = 0.0f;
        for (int n0 = 0; n0 < pieces; n0 += kFlight) {
            float v[kFlight][8];
#pragma unroll
            for (int n = 0; n < kFlight; ++n)
                fetch(n0 + n, v[n]);
#pragma unroll
            for (int n = 0; n < kFlight; ++n)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    sum = fmaf(v[n][k] * f, v[n][k] * f, sum);
        }
        for (int d = 16; d; d >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0)
            sm.warp[warp] = sum;
        __syncthreads();
        if (warp < stacked) {
            float s = 0.0f;
            for (int w = 0; w < rows / kRows; ++w)
                s += sm.warp[warp * (rows / kRows) + w];
            if (lane < ranks) {
                if (CL)
                    far_store(at_rank(smem_u32(&sm.part[rank][warp]), lane), __float_as_uint(s));
                else
                    sm.part[0][warp] = s;
            }
        }
        if (CL) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        if (threadIdx.x < stacked) {
            float s = 0.0f;
            for (int r = 0; r < ranks; ++r)
                s += sm.part[r][threadIdx.x];
            sm.sum[threadIdx.x].sum = s;
            if (!again)
                sm.sum[threadIdx.x].back = b0 + threadIdx.x < a.batch ? back_of(s) : 0;
        }
        // the same in every block of a cluster, which add the same sums
        if (!__syncthreads_or(!again && threadIdx.x < stacked && sm.sum[threadIdx.x & 7].back != 0))
            break;
        back = sm.sum[mine].back;
        if (CL) {  // the parts have been read
            cluster_arrive();
            cluster_wait();
        }
    }
    if (threadIdx.x < stacked) {
        Scale sc = scale_of(sm.sum[threadIdx.x]);
        if (!(sc.unit < INFINITY)) {
            sc = Scale{0, 0.0f};
            sm.bad[threadIdx.x] = 1;
        }
        sm.scale[threadIdx.x] = sc;
    }
    __syncthreads();

    // ---- X_0 = G times a power of two (in two factors, each in range), exactly
    {
        const int e = sm.scale[mine].e;
        const bool out = sm.bad[mine];
        const Pk<2> f0 = pk_all<2>(power_of_two(e / 2)), f1 = pk_all<2>(power_of_two(e - e / 2));
        for (int n0 = 0; n0 < pieces; n0 += kFlight) {
            float v[kFlight][8];
#pragma unroll
            for (int n = 0; n < kFlight; ++n)
                fetch(n0 + n, v[n]);
#pragma unroll
            for (int n = 0; n < kFlight; ++n) {
                if (n0 + n >= pieces)
                    break;
                int r, c;
                where(n0 + n, r, c);
                Pk<2> x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = out ? pk_all<2>(0.0f) : mul_(mul_(Pk<2>::make(v[n][2 * k], v[n][2 * k + 1]), f0), f1);
                float top;
                if (!a.tall) {
                    store8<2>(xs + swizzled(r0 + r, c), S::kX, x, top);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        __half hi, lo;
                        two_terms(x[k / 2].get(k & 1), hi, lo);
                        const uint32_t at = swizzled(r0 + r + k, c);
                        *reinterpret_cast<__half *>(xs + at) = hi;
                        *reinterpret_cast<__half *>(xs + S::kX + at) = lo;
                    }
                }
            }
        }
    }
    fence_async_smem();
    tc_before();
    __syncthreads();
    tc_after();

    const uint32_t tmem = sm.tmem, xa = smem_u32(xs), ea = smem_u32(es), done = smem_u32(&sm.done);
    const int blocks = span >> 6;
    constexpr int kParts = S::kThreads / 128;  // warps that share 32 rows
    const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane, mi = row >> a.log_rows;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const bool real = (row & (rows - 1)) < a.p;
    uint32_t phase = 0;
    // A product added to a sum costs it a rounding towards zero: the 16 of X X^T in
    // 256 columns go to two sums (4 x 128 x 512 normal float: 1.2e-6 off instead of
    // 1.7e-6, 64 x 4000 2.8e-6 instead of 3.2e-6).
    constexpr bool kHalves = PL == 2 && QC == 256;
    auto gram = [&](int col, Pk<2> (&v)[16]) {
        float w[32], u[32];
        tmem_load32(lanes + col, w);
        if (kHalves && blocks > 2)
            tmem_load32(lanes + 128 + col, u);
        tmem_load_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            v[k] = Pk<2>::make(w[2 * k], w[2 * k + 1]);
            if (kHalves && blocks > 2)
                v[k] = add_(v[k], Pk<2>::make(u[2 * k], u[2 * k + 1]));
        }
    };
    auto sums = [&](int col, Pk<2> (&v)[16]) {  // 32 columns
        float w[32];
        tmem_load32(lanes + col, w);
        tmem_load_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k)
            v[k] = Pk<2>::make(w[2 * k], w[2 * k + 1]);
    };
    // A value that fp16 does not hold: told to every block where only this one
    // saw it, and never in the last step after its last barrier (a block may be
    // gone then).
    auto report = [&](int matrix) {
        if (CL) {
            for (int r = 0; r < ranks; ++r)
                far_store(at_rank(smem_u32(&sm.bad[matrix]), r), 1u);
        } else {
            sm.bad[matrix] = 1;
        }
    };
    // Every thread: the products issued last are done, or a wait ran out: then the block
    // goes on without waiting, its results are no numbers, nor those of the blocks that
    // still get something from it (`shared`).
    auto finish = [&](bool shared) {
        if (!mbar_try(done, phase)) {
            const long long start = clock64();
            while (!mbar_try(done, phase) && *(volatile int *)&sm.stop == 0)
                if (clock64() - start > a.wait) {
                    for (int m = 0; m < stacked; ++m) {
                        if (shared)
                            report(m);
                        sm.bad[m] = 1;
                    }
                    __threadfence_block();
                    *(volatile int *)&sm.stop = 1;
                    *(volatile int *)a.status = 1;
                }
            __threadfence_block();
        }
        phase ^= 1;
        tc_after();
    };
    // Eight values of X X^T, columns col and up of row r, to E times its scale:
    // `f` for both, `theta` off the diagonal's element.
    auto e_of = [&](Pk<2> (&v)[4], int r, int col, Pk<2> f, float theta) {
        const int pair = (r & (rows - 1)) < a.p ? r >> 1 : -1;
        const Pk<2> off = r & 1 ? Pk<2>::make(0.0f, -kEs * theta) : Pk<2>::make(-kEs * theta, 0.0f);
        const bool others = rows == 16 && (col >> 4) != (r >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = mul_(v[k], f);
            if (col / 2 + k == pair)
                v[k] = add_(v[k], off);
            if (others)
                v[k] = pk_all<2>(0.0f);
        }
    };
    // A row's matrix has the columns from `block` on; those of the others stay
    // zero in E and B.  Pieces of 32 columns, taken in turn by the warps of a row.
    const int block = (row & ~(rows - 1)) & ~31, pieces32 = rows < 32 ? 1 : rows / 32;
    constexpr int kWide = STACK ? 64 : 128;  // columns that a row of E keeps
    auto e_at = [&](int r, int col) { return swizzled(r, STACK ? col & 63 : col); };
    if (rows < kWide) {
        for (int i = threadIdx.x; i < S::kE / 16; i += S::kThreads)
            reinterpret_cast<uint4 *>(es)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }

    for (int step = 0; step < a.steps; ++step) {
        const float ca = a.coefs[3 * step], cb = a.coefs[3 * step + 1], cc = a.coefs[3 * step + 2];
        const float theta = step == a.steps - 1 ? 1.0f : (step == a.steps - 2 ? 0.5f : 0.0f);
        const bool last = step == a.steps - 1;
        auto unit_of = [&](int matrix) { return step == 0 ? sm.scale[matrix].unit : 1.0f / kXs; };
        auto e_scale = [&](int matrix) {
            const float unit = unit_of(matrix);
            return pk_all<2>(unit * unit * kEs);
        };

        // ---- X X^T
        if (warp == 0 && elect_one()) {
            constexpr uint32_t idesc = mma_desc(128, 128, false);
            if (PL == 2)
                for (int k = 0; k < blocks * 4; ++k) {
                    const uint32_t at = xa + (k >> 2) * 16384 + (k & 3) * 32;
                    tc_mma(tmem, desc_k(at), desc_k(at + S::kX), idesc, k > 0);
                    tc_mma(tmem, desc_k(at + S::kX), desc_k(at), idesc, true);
                }
            for (int k = 0; k < blocks * 4; ++k) {
                const uint32_t at = xa + (k >> 2) * 16384 + (k & 3) * 32;
                const bool second = kHalves && k >= 8;
                tc_mma(second ? tmem + 128 : tmem, desc_k(at), desc_k(at), idesc, second ? k > 8 : (PL == 2 || k > 0));
            }
            tc_commit(done);
        }
        __syncwarp();
        if (CL) {
            // the partial sums in this block's memory: the others have read the
            // last ones, and this block is done with its B
            finish(true);
            const int per = 128 / ranks;
            const int beside = S::kBeside ? S::kE : 0;
            float *const to = reinterpret_cast<float *>(es + beside) + row * 128;
            for (int c = 32 * part; c < 128; c += 32 * kParts) {
                Pk<2> v[16];
                if (blocks) {
                    gram(c, v);
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        v[k] = pk_all<2>(0.0f);
                }
#pragma unroll
                for (int k = 0; k < 32; k += 4)  // pieces of a row rotated by the row: no two lanes on one bank
                    *reinterpret_cast<float4 *>(to + ((c + k + 4 * row) & 127)) =
                        make_float4(v[k / 2].get(0), v[k / 2].get(1), v[k / 2 + 1].get(0), v[k / 2 + 1].get(1));
            }
            cluster_arrive();
            cluster_wait();
            // this block's rows of E: the partial sums in order of rank
            constexpr int kMost = 64 * 16 / S::kThreads;
            Pk<2> v[kMost][4];
            const int pieces = per * 16;
#pragma unroll
            for (int n = 0; n < kMost; ++n) {
                const int piece = threadIdx.x + n * S::kThreads;
                if (piece < pieces) {
                    const int r = piece >> 4, col = (piece & 15) * 8, whole = rank * per + r;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[n][k] = pk_all<2>(0.0f);
                    for (int src = 0; src < ranks; ++src) {
                        const uint32_t from = at_rank(ea + beside + whole * 512, src);
#pragma unroll
                        for (int k = 0; k < 4; k += 2) {
                            const float4 f = far_load(from + ((col + 2 * k + 4 * whole) & 127) * 4);
                            v[n][k] = add_(v[n][k], Pk<2>::make(f.x, f.y));
                            v[n][k + 1] = add_(v[n][k + 1], Pk<2>::make(f.z, f.w));
                        }
                    }
                }
            }
            if (!S::kBeside) {
                cluster_arrive();
                cluster_wait();
            }
#pragma unroll
            for (int n = 0; n < kMost; ++n) {
                const int piece = threadIdx.x + n * S::kThreads;
                if (piece < pieces) {
                    const int r = rank * per + (piece >> 4), col = (piece & 15) * 8;
                    if ((col >> a.log_rows) != (r >> a.log_rows)) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[n][k] = pk_all<2>(0.0f);
                    } else {
                        e_of(v[n], r, col, e_scale(r >> a.log_rows), theta);
                    }
                    float top = 0.0f;
                    uint4 hi, lo;
                    two_terms(v[n][0], hi.x, lo.x, top);
                    two_terms(v[n][1], hi.y, lo.y, top);
                    two_terms(v[n][2], hi.z, lo.z, top);
                    two_terms(v[n][3], hi.w, lo.w, top);
                    if (top > 65504.0f)
                        report(r >> a.log_rows);
                    const uint32_t at = ea + e_at(r, col);
                    // not unrolled: four blocks' stores at once take longer (32 x 128 x 1024
                    // bf16 72 us, one after the other 68)
#pragma unroll 1
                    for (int to_rank = 0; to_rank < ranks; ++to_rank) {
                        const uint32_t far = at_rank(at, to_rank);
                        far_store(far, hi);
                        if (PL == 2)
                            far_store(far + S::kPlane, lo);
                    }
                }
            }
            tc_before();
            cluster_arrive();
            cluster_wait();
            fence_async_smem();
        } else {
            finish(true);
            float top = 0.0f;
            const Pk<2> scale_e = e_scale(mi);
            for (int n = part; n < pieces32; n += kParts) {
                const int c = block + n * 32;
                Pk<2> v[16];
                gram(c, v);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    Pk<2> w[4] = {v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
                    e_of(w, row, c + 8 * g, scale_e, theta);
                    store8<PL>(es + e_at(row, c + 8 * g), S::kPlane, w, top);
                }
            }
            if (top > 65504.0f)
                report(mi);
            fence_async_smem();
        }
        tc_before();
        __syncthreads();

        // ---- E E, and B in E's place
        if (warp == 0 && elect_one()) {
            tc_after();
            constexpr uint32_t idesc = mma_desc(128, 128, false);
            if (PL == 2)
                for (int k = 0; k < kWide / 16; ++k) {
                    const uint32_t at = ea + (k >> 2) * 16384 + (k & 3) * 32;
                    tc_mma(tmem, desc_k(at), desc_k(at + S::kPlane), idesc, k > 0);
                    tc_mma(tmem, desc_k(at + S::kPlane), desc_k(at), idesc, true);
                }
            for (int k = 0; k < kWide / 16; ++k) {
                const uint32_t at = ea + (k >> 2) * 16384 + (k & 3) * 32;
                tc_mma(tmem, desc_k(at), desc_k(at), idesc, PL == 2 || k > 0);
            }
            tc_commit(done);
        }
        __syncwarp();
        finish(!last);
        const float b0c = (cb + 2.0f * cc * theta) * (kBs / kEs), b1c = cc * (kBs / kEs / kEs);
        float top = 0.0f;
        for (int n = part; n < pieces32; n += kParts) {
            const int c = block + n * 32;
            Pk<2> v[16];
            sums(c, v);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                char *at = es + e_at(row, c + 8 * g);
                Pk<2> e[4];
                load8<PL>(at, S::kPlane, e);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    e[k] = fma_(pk_all<2>(b0c), e[k], mul_(pk_all<2>(b1c), v[4 * g + k]));
                store8<PL>(at, S::kPlane, e, top);
            }
        }
        if (top > 65504.0f)
            sm.bad[mi] = 1;  // every block has this B
        fence_async_smem();
        tc_before();
        __syncthreads();

        // ---- B X, and the next X in X's place
        if (warp == 0 && elect_one()) {
            tc_after();
            // STACK: X's blocks of 64 columns, each for the upper and the lower 64 rows
            constexpr uint32_t idesc = mma_desc(128, STACK ? 2 * QC : QC, true);
            constexpr uint32_t next = STACK ? 8192 : 16384;
            if (PL == 2)
                for (int k = 0; k < kWide / 16; ++k) {
                    const uint32_t at = ea + (k >> 2) * 16384 + (k & 3) * 32, xt = xa + k * 2048;
                    tc_mma(tmem, desc_k(at), desc_mn(xt + S::kX, next), idesc, k > 0);
                    tc_mma(tmem, desc_k(at + S::kPlane), desc_mn(xt, next), idesc, true);
                }
            for (int k = 0; k < kWide / 16; ++k) {
                const uint32_t at = ea + (k >> 2) * 16384 + (k & 3) * 32, xt = xa + k * 2048;
                tc_mma(tmem, desc_k(at), desc_mn(xt, next), idesc, PL == 2 || k > 0);
            }
            tc_commit(done);
        }
        __syncwarp();
        finish(!last);
        const float x0 = ca + theta * (cb + theta * cc), unit = unit_of(mi);
        const float scale = last ? unit : unit * kXs;
        const long long b = b0 + mi;
        const int i = row & (rows - 1);
        const bool bad = last && sm.bad[mi];
        T *const out = (T *)a.X + b * a.xb + (a.tall ? i + c0 * a.xr : i * a.xr + c0);
        top = 0.0f;
        const Pk<2> sx = pk_all<2>(scale * x0), sb = pk_all<2>(scale * (1.0f / kBs));
        for (int c = 32 * part; c < span; c += 32 * kParts) {
            Pk<2> v[16];
            sums(STACK ? (c >> 6) * 128 + (row & 64) + (c & 63) : c, v);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                char *at = xs + swizzled(row, c + 8 * g);
                Pk<2> x[4];
                load8<2>(at, S::kX, x);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = fma_(sx, x[k], mul_(sb, v[4 * g + k]));
                if (!last) {
                    store8<2>(at, S::kX, x, top);
                } else if (real && b < a.batch) {
                    T *to = out + (a.tall ? (long long)(c + 8 * g) * a.xr : (long long)(c + 8 * g));
                    const long long by = a.tall ? a.xr : 1;
                    Row8<T> y;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        store_last(&y.v[k], bad ? nanf("") : x[k / 2].get(k & 1));
                    if (a.vector_out && c + 8 * g + 8 <= width) {
                        *reinterpret_cast<Row8<T> *>(to) = y;
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (c + 8 * g + k < width)
                                to[k * by] = y.v[k];
                    }
                }
            }
        }
        if (!last && top > 65504.0f)
            report(mi);
        fence_async_smem();
        tc_before();
        __syncthreads();
        tc_after();
    }
    if (warp == 0) {
        if (elect_one() && sm.stop) {  // the last products may still run
            tc_commit(smem_u32(&sm.drained));
            mbar_wait(smem_u32(&sm.drained), 0);
        }
        __syncwarp();
        tmem_free(tmem, S::kCols);
    }
}

}  // namespace
}  // namespace bstq
