// Gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t, its gradients and
// its single-token form: kernels and entry points.
//
// Both directions are one pass over memory.  A tile is 64 channels (a pair to a
// lane) by W * L tokens (L to each of W = 8 or 11 warps).  Per tile these warps
//   1. turn r into q_t = 1 - a_t and run their L tokens from a zero state, which
//      gives each warp's map h -> h + (v - Q h), Q = 1 - exp(-sum of z) (the
//      gradients: h -> A h + v, in the form of decay());
//   2. wait for the state that enters their tokens, run them again from it and
//      leave h in place of x in shared memory;
// each copies its own rows in and out (TMA, two stages: the next tile's rows
// arrive while this one's state is awaited), and one more warp finds the state
// that enters the tile and publishes what the tiles after it need.
// That state comes together in a fixed order, so that equal inputs give equal
// bits: tiles of a channel form groups; the last tile of a group publishes the
// state after it, and a tile applies the maps of the tiles before it in its own
// group to the state after the last group (the maps of four tiles joined into one
// by the last of the four).  Tiles publish their maps as soon as they have them,
// so only the group states wait for each other.  Where there are as many tiles of
// channels as blocks, a tile's predecessor is a whole round older and a group is
// one tile (one word a channel to read); with fewer, several tiles of a channel
// run at once and groups of 16 divide the waits by as much.
// Maps and states carry their own mark of being there (the workspace starts as a
// NaN that no sum gives), so a wait is one round trip to L2.
// The launch is cooperative: every block is resident and takes its tiles in
// ascending order, a tile waits for lower ones only, and so every wait ends.
//
// Rounding: a state is updated as h + q (x - h), never as a product with a decay
// that was rounded near one, and maps carry Q = 1 - A for the same reason: over
// 32768 tokens a product of float decays drifts by 1e-4, this form by 3e-7.  That is
// relative to x and h; the gradients are products with a, s and 1 - s, which may be
// small, and keep the digits of those too.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <stdint.h>

#include <atomic>

#include "../../include/bstq.h"
#include "bstq_common.h"
#include "bstq_pack.cuh"
#include "bstq_tensor.cuh"

namespace bstq {
namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

struct Seq {
    long long sb, st;  // element strides of the batch and the time axis
};

__device__ __forceinline__ float ex2(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
constexpr float kLog2e = 1.44269504f;

// 1 - exp(-z) for 0 <= z < 3/4 to two units in the last place: z times the Chebyshev
// interpolant of (1 - exp(-z)) / z of degree 5 (off by 3.3e-8 at most).
template <int V>
__device__ __forceinline__ Pk<V> near_zero(Pk<V> z)
{
    Pk<V> f = pk_all<V>(-0.0010119646f);
    f = fma_(f, z, pk_all<V>(0.0080331592f));
    f = fma_(f, z, pk_all<V>(-0.0415530764f));
    f = fma_(f, z, pk_all<V>(0.1666469872f));
    f = fma_(f, z, pk_all<V>(-0.4999987483f));
    f = fma_(f, z, pk_all<V>(1.0f));
    return mul_(f, z);
}
template <int V>
__device__ __forceinline__ Pk<V> exp_minus(Pk<V> z)
{
    const Pk<V> y = mul_(z, pk_all<V>(-kLog2e));
    float e[V];
#pragma unroll
    for (int k = 0; k < V; ++k)
        e[k] = ex2(y.get(k));
    return pk<V>(e);
}

// 1 - exp(-z) for z >= 0: from 3/4 on one minus the exponential.
template <int V>
__device__ __forceinline__ Pk<V> one_minus_exp(Pk<V> z)
{
    const Pk<V> f = near_zero<V>(z), g = fma_(exp_minus<V>(z), pk_all<V>(-1.0f), pk_all<V>(1.0f));
    float out[V];
#pragma unroll
    for (int k = 0; k < V; ++k)
        out[k] = z.get(k) < 0.75f ? f.get(k) : g.get(k);
    return pk<V>(out);
}

// The gradients need a = exp(-z) and 1 - a each to its own last digits: a is a
// factor of dr, drate and dh0 (1 - (1 - a) in floats is off by 2.6e-2 of a at z = 15
// and zero at 18), 1 - a one of dx.  One number holds both: -(1 - a) for z < 3/4,
// else a.  It is the smaller of the two (at most 0.53), the other is one minus it,
// and the sign bit tells which.
__device__ __forceinline__ bool is_loss(float n) { return __float_as_int(n) < 0; }
__device__ __forceinline__ Pk<2> decay(Pk<2> z)
{
    const Pk<2> f = near_zero<2>(z), e = exp_minus<2>(z);
    return Pk<2>::make(z.get(0) < 0.75f ? -f.get(0) : e.get(0), z.get(1) < 0.75f ? -f.get(1) : e.get(1));
}
// g where n is a loss, else zero: a g = n g + whole, (1 - a) g = (g - whole) - n g.
__device__ __forceinline__ Pk<2> whole(Pk<2> n, Pk<2> g)
{
    return Pk<2>::make(is_loss(n.get(0)) ? g.get(0) : 0.0f, is_loss(n.get(1)) ? g.get(1) : 0.0f);
}
__device__ __forceinline__ float kept(float n, float g) { return fmaf(n, g, is_loss(n) ? g : 0.0f); }  // a g
__device__ __forceinline__ Pk<2> kept(Pk<2> n, Pk<2> g) { return fma_(n, g, whole(n, g)); }

// s = sigma(r) from e = exp(-r): where that overflows, 0.
template <int V>
__device__ __forceinline__ Pk<V> sigma_of(Pk<V> e)
{
    const Pk<V> d = add_(e, pk_all<V>(1.0f));
    float s[V];
#pragma unroll
    for (int k = 0; k < V; ++k)
        s[k] = rcp(d.get(k));
    return pk<V>(s);
}
template <int V>
__device__ __forceinline__ Pk<V> sigma(Pk<V> r)
{
    return sigma_of<V>(exp_minus<V>(r));
}
// 1 - s = e s to its own digits: 1 - s from a rounded s is off by 9e-3 at r = 12 and
// zero at 17.  Where e overflows and s is zero their product is no number, and 1 - s one.
__device__ __forceinline__ Pk<2> one_minus_sigma(Pk<2> s, Pk<2> e)
{
    const Pk<2> o = mul_(e, s);
    return Pk<2>::make(fminf(o.get(0), 1.0f), fminf(o.get(1), 1.0f));
}

// A pair of neighbouring values in memory.
__device__ __forceinline__ Pk<2> get2(const float *p)
{
    Pk<2> v;
    v.v = *reinterpret_cast<const unsigned long long *>(p);
    return v;
}
__device__ __forceinline__ Pk<2> get2(const __nv_bfloat16 *p)
{
    const uint32_t u = *reinterpret_cast<const uint32_t *>(p);
    return Pk<2>::make(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ Pk<2> get2(const __half *p)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(p));
    return Pk<2>::make(f.x, f.y);
}
__device__ __forceinline__ void put2(float *p, Pk<2> v) { *reinterpret_cast<unsigned long long *>(p) = v.v; }
__device__ __forceinline__ void put2(__nv_bfloat16 *p, Pk<2> v)
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.get(0), v.get(1));
}
__device__ __forceinline__ void put2(__half *p, Pk<2> v)
{
    *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(v.get(0), v.get(1));
}

__device__ __forceinline__ int length_of(const int32_t *lengths, long long b, long long time)
{
    if (!lengths)
        return (int)time;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > time ? (int)time : n);
}

struct RecurArgs {
    long long batch, time, dim;
    const void *x, *r, *h_in, *dh;
    const float *rate, *h0, *dhT;
    const int32_t *lengths;
    void *h, *dx, *dr;
    float *hT, *dh0, *drate, *part;
    Seq sx, sr, sh, sdh, sdx, sdr;
    // tiles: `ranks` along time (counted from the end for the gradients) for
    // each of `chains` = batch * cols tiles of channels; a block goes from one
    // tile to its next by step_rank ranks and step_chain chains
    int ranks, cols, chains, step_rank, step_chain, group;
    // (v, Q or, for the gradients, decay()'s number): [chain][rank][64], then of four
    // tiles, [chain][rank / 4][64]
    unsigned long long *maps;
    unsigned long long *states;  // two channels to a word, [chain][group][32]
    int *status;
    long long wait;  // cycles after which a wait gives up
};

struct RecurMaps {  // TMA: inputs x, r (h, dh), outputs h or dx, dr
    CUtensorMap in[4], out[2];
};

constexpr int kChannels = 64;
constexpr int kMaxGroup = 16;
constexpr uint32_t kUnset = 0xffffffffu;

// Warps of a tile and tokens of a lane: eight warps and three blocks to an SM
// forward; the gradients, with four tensors and more registers, do better in two
// blocks of eleven warps (8 x 2048 x 4096 bf16 175 us against 186 with eight in three
// blocks, 192 with ten and 184 with twelve in two; 1 x 32768 x 1024 143 against 147,
// 153 and 142).
template <typename T, bool GRAD>
struct Tile {
    static constexpr int W = GRAD ? 11 : 8, BLOCKS = GRAD ? 2 : 3;
    static constexpr int THREADS = 32 * (W + 1);
    static constexpr int L = (sizeof(T) == 2 ? 16 : 8) / (GRAD ? 2 : 1);
    static constexpr int TOK = W * L;
    static constexpr int IN = GRAD ? 4 : 2, OUT = GRAD ? 2 : 1;
    static constexpr int BYTES = TOK * kChannels * (int)sizeof(T);
    static constexpr int STAGE = IN * BYTES;
    static constexpr int ROWS = BYTES / W;  // a warp's share of one tensor
};

// Barriers: `full` a warp's rows are there; `ready` every warp has its map;
// `entered` the state that enters the tile is there.  Maps and states are there
// for two tiles in turn: a warp may be one tile ahead of another.
template <int W>
struct alignas(128) TileShared {
    float q[2][W][kChannels], v[2][W][kChannels];
    float enter[2][kChannels];
    float sums[W][kChannels];  // of dz s
    uint64_t full[2][W], ready[2], entered[2];
    int stop;
};
template <typename T, bool GRAD>
constexpr int tile_smem()
{
    return (int)sizeof(TileShared<Tile<T, GRAD>::W>) + 2 * Tile<T, GRAD>::STAGE;
}
static_assert(3 * (tile_smem<float, false>() + 1024) <= 228 * 1024 && 2 * (tile_smem<float, true>() + 1024) <= 228 * 1024,
              "the blocks of an SM");

// A wait that ends: with its barrier (true), after two seconds, or when another ended so
// (false).  From then on the block's barriers may complete too early, for its warps go
// on arriving.  But `stop` is set before, and who waits for such an arrival sees it: so a
// thread that reads stop == 0 after a wait has what it waited for, and one that reads 1
// has no number, gives NaN on and writes nothing that others may still read.
template <int W>
__device__ __forceinline__ bool wait_for(TileShared<W> &sm, uint64_t &bar, uint32_t parity, const RecurArgs &a)
{
    const uint32_t at = smem_u32(&bar);
    if (mbar_try(at, parity))
        return true;
    const long long start = clock64();
    while (!mbar_try(at, parity)) {
        if (*(volatile int *)&sm.stop)
            return false;
        if (clock64() - start > a.wait) {
            *(volatile int *)&sm.stop = 1;
            *(volatile int *)a.status = 1;
        }
    }
    return true;
}
template <int W>
__device__ __forceinline__ bool stopped(const TileShared<W> &sm)
{
    return *(const volatile int *)&sm.stop != 0;
}
__device__ __forceinline__ float no_number() { return __int_as_float(0x7fffffff); }

__device__ __forceinline__ unsigned long long load_mark(const unsigned long long *p)
{
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ void load_marks(const unsigned long long *p, unsigned long long &a, unsigned long long &b)
{
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "l"(p));
}
__device__ __forceinline__ uint32_t marked(float v)  // v's bits; any NaN as one that is not kUnset
{
    return v != v ? 0x7fffffffu : __float_as_uint(v);
}
__device__ __forceinline__ void publish_map(unsigned long long *p, float q, float v)
{
    const unsigned long long bits = ((unsigned long long)marked(q) << 32) | __float_as_uint(v);
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(bits) : "memory");
}
// The states of a lane's two channels, written and read as one word: accesses of
// different sizes to one place are not ordered by the memory model.
__device__ __forceinline__ void publish_states(unsigned long long *p, float a, float b)
{
    const unsigned long long bits = ((unsigned long long)marked(b) << 32) | marked(a);
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(bits) : "memory");
}

// A map h -> h + (v - q h) of each of a lane's two channels.  FINE (the gradients):
// h -> a h + v with a = 1 - q to its own digits, passed on as decay()'s number.
template <bool FINE>
struct Map2 {
    float q[2] = {0.0f, 0.0f}, v[2] = {0.0f, 0.0f}, a[2] = {1.0f, 1.0f};
    static __device__ __forceinline__ float none() { return FINE ? -0.0f : 0.0f; }
    __device__ __forceinline__ float passed(int c) const { return !FINE ? q[c] : (q[c] < 0.5f ? -q[c] : a[c]); }
    __device__ __forceinline__ float of(int c, float h) const
    {
        return FINE ? kept(passed(c), h) + v[c] : h + (v[c] - q[c] * h);
    }
    __device__ __forceinline__ void then(const float (&m)[2], const float (&mv)[2])
    {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (FINE) {
                const bool loss = is_loss(m[c]);
                const float mq = loss ? -m[c] : 1.0f - m[c];
                v[c] = kept(m[c], v[c]) + mv[c];
                q[c] += mq - mq * q[c];
                a[c] *= loss ? 1.0f + m[c] : m[c];
            } else {
                v[c] += mv[c] - m[c] * v[c];
                q[c] += m[c] - m[c] * q[c];
            }
        }
    }
    __device__ __forceinline__ void then(const Map2 &next)
    {
        const float m[2] = {next.passed(0), next.passed(1)};
        then(m, next.v);
    }
};

// Reads up to three published maps in a row (`n` of them) and joins them; false
// while one is missing.
template <bool FINE>
__device__ __forceinline__ bool read_maps(const unsigned long long *at, int n, Map2<FINE> &m)
{
    m = Map2<FINE>{};
    if (n <= 0)
        return true;
    unsigned long long w[3][2];
#pragma unroll
    for (int i = 0; i < 3; ++i)
        load_marks(at + (i < n ? i : n - 1) * kChannels, w[i][0], w[i][1]);
    bool there = true;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        float q[2], v[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t mark = (uint32_t)(w[i][c] >> 32);
            there = there && mark != kUnset;
            q[c] = i < n ? __uint_as_float(mark) : Map2<FINE>::none();
            v[c] = i < n ? __uint_as_float((uint32_t)w[i][c]) : 0.0f;
        }
        m.then(q, v);
    }
    return __all_sync(0xffffffffu, there);
}

// The last warp's part in a tile, with the channels 2 lane and 2 lane + 1:
// leaves the entering state for the others, publishes the tile's map (or that of
// its four tiles, or the state after its group) and returns the state after the
// tile.  `first` is the channels' first tile, `last` their last.  `between` runs
// when every warp has its map.  `dead`: this thread has no numbers any more.
template <bool GRAD, int W, typename F>
__device__ __forceinline__ void chain(const RecurArgs &a, TileShared<W> &sm, int slot, uint32_t phase, int chain_id, int rank,
                                      int first, int last, const float *start, const bool (&on)[2], F between,
                                      float (&enter)[2], float (&after)[2], bool &dead)
{
    const int lane = threadIdx.x & 31;
    const int group = rank / a.group, groups = (a.ranks + a.group - 1) / a.group;
    const int from = group * a.group > first ? group * a.group : first;
    const int four = a.group == 1 ? rank : rank & ~3;  // this tile's four begin here
    const int single = four > from ? four : from;
    const bool grouped = from > first;
    const long long at = (long long)chain_id * a.ranks;
    unsigned long long *states = a.states + (long long)chain_id * groups * (kChannels / 2) + lane;
    unsigned long long *singles = a.maps + at * kChannels + 2 * lane;
    unsigned long long *fours = a.maps + ((long long)a.chains * a.ranks + (long long)chain_id * ((a.ranks + 3) / 4)) * kChannels + 2 * lane;
    constexpr bool EARLY = !GRAD;
    Map2<GRAD> own, near;
    bool have_near = single == rank, entered = false, mine = false;
    const uint32_t ready = smem_u32(&sm.ready[slot]);
    auto leave = [&] {
        if (!dead)
            *reinterpret_cast<float2 *>(&sm.enter[slot][2 * lane]) = make_float2(enter[0], enter[1]);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_u32(&sm.entered[slot]));
    };
    auto publish = [&] {
        if (rank >= last)
            return;
        if (rank - four < 3) {
            publish_map(singles + (long long)rank * kChannels, own.passed(0), own.v[0]);
            publish_map(singles + (long long)rank * kChannels + 1, own.passed(1), own.v[1]);
        } else if (rank % a.group < a.group - 1) {
            Map2<GRAD> all = near;
            all.then(own);
            publish_map(fours + (long long)(rank / 4) * kChannels, all.passed(0), all.v[0]);
            publish_map(fours + (long long)(rank / 4) * kChannels + 1, all.passed(1), all.v[1]);
        }
    };
    const bool maps = a.group > 1;
    long long t0 = 0;
    do {
        if (!have_near && read_maps(singles + (long long)single * kChannels, rank - single, near)) {
            have_near = true;
            if (mine && !dead && rank - four == 3)
                publish();
        }
        if (!entered) {
            bool there = true;
            enter[0] = enter[1] = 0.0f;
            if (grouped) {
                const unsigned long long s = load_mark(states + (long long)(group - 1) * (kChannels / 2));
                there = (uint32_t)s != kUnset && (uint32_t)(s >> 32) != kUnset;
                enter[0] = __uint_as_float((uint32_t)s), enter[1] = __uint_as_float((uint32_t)(s >> 32));
            } else if (start) {
                enter[0] = on[0] ? start[0] : 0.0f;
                enter[1] = on[1] ? start[1] : 0.0f;
            }
            Map2<GRAD> far;
            if (maps)
                there = read_maps(fours + (long long)(from / 4) * kChannels, rank / 4 - from / 4, far) && there;
            if (__all_sync(0xffffffffu, there) && have_near) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    enter[c] = near.of(c, far.of(c, enter[c]));
                entered = true;
                if (EARLY || mine)
                    leave();
            }
        }
        // with the entering state known there is nothing to do but sleep
        if (!mine && __all_sync(0xffffffffu, entered ? mbar_try(ready, phase) : mbar_test(ready, phase))) {
            mine = true;
            dead = stopped(sm) || dead;
            between();
            if (!EARLY && entered)
                leave();
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float2 wq = *reinterpret_cast<const float2 *>(&sm.q[slot][w][2 * lane]);
                const float2 wv = *reinterpret_cast<const float2 *>(&sm.v[slot][w][2 * lane]);
                const float mq[2] = {wq.x, wq.y}, mv[2] = {wv.x, wv.y};
                own.then(mq, mv);
            }
            if (maps && !dead && (have_near || rank - four < 3))
                publish();
        }
        if (entered && mine)
            break;
        if (t0 == 0)
            t0 = clock64();
        if (clock64() - t0 > a.wait) {
            *(volatile int *)&sm.stop = 1;
            *(volatile int *)a.status = 1;
        }
    } while (__any_sync(0xffffffffu, !stopped(sm)));
    if (!entered || !mine)
        dead = true;
    if (dead) {  // told to those who wait for the tile, too
        enter[0] = enter[1] = after[0] = after[1] = no_number();
        const int block = rank / 4;
        for (int c = 0; c < 2 && maps; ++c) {
            publish_map(singles + (long long)rank * kChannels + c, no_number(), no_number());
            publish_map(fours + (long long)block * kChannels + c, no_number(), no_number());
        }
        publish_states(states + (long long)group * (kChannels / 2), no_number(), no_number());
        return;
    }
    after[0] = own.of(0, enter[0]);
    after[1] = own.of(1, enter[1]);
    if (rank < last && rank % a.group == a.group - 1)
        publish_states(states + (long long)group * (kChannels / 2), after[0], after[1]);
}

__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}

// Where a block is: its tile of channels, its rank, and what the sequence's
// length makes of it.
struct Place {
    int rank, ch;
    int b, j0, n;
    int first, last;  // the ranks that hold tokens of the sequence
};
template <bool GRAD, int TOK>
__device__ __forceinline__ Place place_of(const RecurArgs &a, int rank, int ch)
{
    Place p;
    p.rank = rank, p.ch = ch;
    p.b = ch / a.cols;
    p.j0 = (ch - p.b * a.cols) * kChannels;
    p.n = length_of(a.lengths, p.b, a.time);
    const int held = p.n ? (p.n - 1) / TOK : 0;
    p.first = GRAD ? a.ranks - 1 - held : 0;
    p.last = GRAD ? a.ranks - 1 : held;
    return p;
}
__device__ __forceinline__ void next_place(const RecurArgs &a, int &rank, int &ch)
{
    rank += a.step_rank;
    ch += a.step_chain;
    if (ch >= a.chains)
        ch -= a.chains, ++rank;
}
__device__ __forceinline__ bool holds(const Place &p) { return p.rank >= p.first && p.rank <= p.last; }

// One lane's L tokens in a tile, MASK: some of them past the end.  TMA: results
// go to shared memory in place of x (and r); otherwise straight to memory.
template <typename T, bool GRAD, bool MASK, bool TMA>
struct LaneRun {
    using S = Tile<T, GRAD>;
    static constexpr int L = S::L;
    const RecurArgs &a;
    T *tile;  // the stage, at this lane's channels
    const Place &p;
    int warp, lane;
    Pk<2> q[L], e[GRAD ? L : 1];  // 1 - a; for the gradients decay()'s numbers, and exp(-r)

    // the row of token t in the tile, and the token itself; for the gradients
    // t counts backwards
    __device__ __forceinline__ int row(int t) const { return GRAD ? S::TOK - 1 - (warp * L + t) : warp * L + t; }
    __device__ __forceinline__ int token(int t) const
    {
        return (GRAD ? a.ranks - 1 - p.rank : p.rank) * S::TOK + row(t);
    }
    __device__ __forceinline__ T *at(int k, int t) const { return tile + (k * S::TOK + row(t)) * kChannels; }

    __device__ __forceinline__ void first(Pk<2> rate, Pk<2> &z, Pk<2> &v)
    {
        z = v = pk_all<2>(0.0f);
#pragma unroll
        for (int t = 0; t < L; ++t) {
            if (MASK && token(t) >= p.n) {
                q[t] = pk_all<2>(0.0f);
                continue;
            }
            const Pk<2> er = exp_minus<2>(get2(at(1, t))), zt = mul_(rate, sigma_of<2>(er));
            if (GRAD)
                e[GRAD ? t : 0] = er;
            q[t] = GRAD ? decay(zt) : one_minus_exp<2>(zt);
            z = add_(z, zt);
            if (GRAD) {
                v = add_(v, get2(at(3, t)));
                // as in whole(), by the comparison that decay() has made
                const Pk<2> w = Pk<2>::make(zt.get(0) < 0.75f ? v.get(0) : 0.0f, zt.get(1) < 0.75f ? v.get(1) : 0.0f);
                v = fma_(q[t], v, w);
            } else {
                v = fma_(q[t], sub_<2>(get2(at(0, t)), v), v);
            }
        }
    }
    // one result: k'th output at token t
    __device__ __forceinline__ void out(int k, int t, Pk<2> v) const
    {
        if (TMA) {
            put2(at(k, t), v);
        } else if (token(t) < a.time) {
            const Seq &sq = GRAD ? (k ? a.sdr : a.sdx) : a.sh;
            T *to = (T *)(GRAD ? (k ? a.dr : a.dx) : a.h) + p.b * sq.sb + token(t) * sq.st;
            const int j = p.j0 + 2 * lane;
            if (j < a.dim)
                to[j] = from_f<T>(v.get(0));
            if (j + 1 < a.dim)
                to[j + 1] = from_f<T>(v.get(1));
        }
    }
    __device__ __forceinline__ void forward(Pk<2> h) const
    {
#pragma unroll
        for (int t = 0; t < L; ++t) {
            if (MASK && token(t) >= p.n) {
                out(0, t, pk_all<2>(0.0f));
                continue;
            }
            h = fma_(q[t], sub_<2>(get2(at(0, t)), h), h);
            out(0, t, h);
        }
    }
    __device__ __forceinline__ Pk<2> backward(Pk<2> g, Pk<2> rate, Pk<2> h0) const
    {
        Pk<2> sum = pk_all<2>(0.0f);
#pragma unroll
        for (int t = 0; t < L; ++t) {
            if (MASK && token(t) >= p.n) {
                out(0, t, pk_all<2>(0.0f));
                out(1, t, pk_all<2>(0.0f));
                continue;
            }
            g = add_(g, get2(at(3, t)));
            const Pk<2> w = whole(q[t], g), gx = sub_(sub_(g, w), mul_(q[t], g));
            g = fma_(q[t], g, w);
            Pk<2> before = get2(at(2, t));
            if (t == L - 1 && token(t) == 0)
                before = h0;
            const Pk<2> dz = mul_(g, sub_<2>(get2(at(0, t)), before));
            // the gate once more: its registers would not fit beside e
            const Pk<2> er = e[GRAD ? t : 0], s = sigma_of<2>(er);
            const Pk<2> ds = mul_(dz, s);  // summed: drate; times lambda (1 - s): dr
            sum = add_(sum, ds);
            out(0, t, gx);
            out(1, t, mul_(mul_(ds, rate), one_minus_sigma(s, er)));
        }
        return sum;
    }
};

// One warp's rows of a tile by its own loads (rows that TMA cannot copy).
template <typename T, bool GRAD>
__device__ __forceinline__ void load_rows(const RecurArgs &a, const Place &p, T *stage, int warp, int lane)
{
    using S = Tile<T, GRAD>;
    const int tok0 = (GRAD ? a.ranks - 1 - p.rank : p.rank) * S::TOK;
    const int row0 = GRAD ? S::TOK - (warp + 1) * S::L : warp * S::L;
#pragma unroll
    for (int k = 0; k < S::IN; ++k) {
        const Seq &sq = k == 0 ? a.sx : (k == 1 ? a.sr : (k == 2 ? a.sh : a.sdh));
        const T *src = (const T *)(k == 0 ? a.x : (k == 1 ? a.r : (k == 2 ? a.h_in : a.dh))) + p.b * sq.sb + p.j0 + lane;
        T *dst = stage + (k * S::TOK + row0) * kChannels + lane;
#pragma unroll
        for (int t = 0; t < S::L; ++t) {
            const int tok = tok0 + row0 + t, from = k == 2 ? tok - 1 : tok;
            const bool in = tok < p.n && from >= 0;
            const T *at = src + (in ? (long long)from * sq.st : 0);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const bool on = in && p.j0 + lane + 32 * c < a.dim;
                if constexpr (sizeof(T) == 4)
                    copy4(smem_u32(dst + t * kChannels + 32 * c), on ? (const void *)(at + 32 * c) : (const void *)a.rate, on);
                else
                    dst[t * kChannels + 32 * c] = on ? at[32 * c] : from_f<T>(0.0f);
            }
        }
    }
    if constexpr (sizeof(T) == 4)
        asm volatile("cp.async.commit_group;" ::: "memory");
}

// The same by TMA, a box of L rows per tensor.
template <typename T, bool GRAD>
__device__ __forceinline__ void tma_rows(const RecurArgs &a, const RecurMaps &maps, const Place &p, T *stage, int warp,
                                         uint64_t &full)
{
    using S = Tile<T, GRAD>;
    const int tok0 = (GRAD ? a.ranks - 1 - p.rank : p.rank) * S::TOK;
    const int row0 = GRAD ? S::TOK - (warp + 1) * S::L : warp * S::L;
    const uint32_t at = smem_u32(stage + row0 * kChannels), bar = smem_u32(&full);
    mbar_expect(bar, S::IN * S::ROWS);
#pragma unroll
    for (int k = 0; k < S::IN; ++k)
        tma_load(at + k * S::BYTES, &maps.in[k], bar, p.j0, tok0 + row0 - (k == 2 ? 1 : 0), p.b);
}

template <bool B>
struct Flag {
    static constexpr bool value = B;
};

template <typename T, bool GRAD, bool TMA>
__global__ void __launch_bounds__(Tile<T, GRAD>::THREADS, Tile<T, GRAD>::BLOCKS) recur_kernel(RecurArgs a, const __grid_constant__ RecurMaps maps)
{
    using S = Tile<T, GRAD>;
    extern __shared__ __align__(128) char raw[];
    using Shared = TileShared<S::W>;
    Shared &sm = *reinterpret_cast<Shared *>(raw);
    char *stages = raw + sizeof(Shared);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0)
            *(volatile int *)a.status = 0;
        for (int s = 0; s < 2; ++s) {
            for (int w = 0; w < S::W; ++w)
                mbar_init(smem_u32(&sm.full[s][w]), 1);
            mbar_init(smem_u32(&sm.ready[s]), S::W);
            mbar_init(smem_u32(&sm.entered[s]), 1);
        }
        sm.stop = 0;
        mbar_init_fence();
    }
    __syncthreads();
    int rank = blockIdx.x / a.chains, ch = blockIdx.x - rank * a.chains;
    uint32_t phase = 0;

    if (warp == S::W) {
        const float *from = GRAD ? a.dhT : a.h0;
        float *to = GRAD ? a.dh0 : a.hT;
        // the tile before, whose sums of dz s are whole once every warp has come
        // to the next one
        Place before{};
        bool any = false, dead = false;
        auto sums = [&] {
            if (GRAD && any)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int j = before.j0 + 2 * lane + k;
                    float sum = dead ? no_number() : 0.0f;
                    if (holds(before))
#pragma unroll
                        for (int w = 0; w < S::W; ++w)
                            sum += sm.sums[w][2 * lane + k];
                    if (j < a.dim)
                        a.part[((long long)before.b * a.ranks + before.rank) * a.dim + j] = sum;
                }
        };
        int slot = 0;
        for (; rank < a.ranks; slot ^= 1) {
            const Place c = place_of<GRAD, S::TOK>(a, rank, ch);
            if (holds(c)) {
                const bool on[2] = {c.j0 + 2 * lane < a.dim, c.j0 + 2 * lane + 1 < a.dim};
                const long long at = (long long)c.b * a.dim + c.j0 + 2 * lane;
                float enter[2], after[2];
                // the sums have one place: no warp gets to its next ones before they are read
                chain<GRAD, S::W>(a, sm, slot, phase, c.ch, c.rank, c.first, c.last, from ? from + at : nullptr, on, sums,
                                  enter, after, dead);
                if (c.rank == c.last && to)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (on[k])
                            to[at + k] = c.n ? after[k] : enter[k];
            } else {
                wait_for(sm, sm.ready[slot], phase, a);  // keeps the phases in step
                dead = stopped(sm) || dead;
                sums();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm.entered[slot]));
            }
            before = c;
            any = true;
            next_place(a, rank, ch);
            phase ^= slot;
        }
        if (GRAD) {
            wait_for(sm, sm.ready[slot], phase, a);
            dead = stopped(sm) || dead;
            sums();
        }
        return;
    }

    uint32_t loaded[2] = {0, 0};
    auto rates = [&](const Place &p) {
        float v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j = p.j0 + 2 * lane + k;
            v[k] = j < a.dim ? a.rate[j] : 0.0f;
            v[k] = v[k] <= 0.0f ? 0.0f : v[k];  // no zero with a sign
        }
        return pk<2>(v);
    };
    // whether this thread has had all that it waited for, and the next tile's rows were
    // asked for
    bool ok = true, asked = false;
    // a warp's rows of a tile into a stage that holds its own results of the
    // tile before last, stored by then
    auto load = [&](const Place &p, int slot) {
        asked = ok && holds(p);
        if (!holds(p))
            return;
        T *stage = (T *)(stages + slot * S::STAGE);
        if (!TMA) {
            load_rows<T, GRAD>(a, p, stage, warp, lane);
        } else if (lane == 0 && asked) {
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            tma_rows<T, GRAD>(a, maps, p, stage, warp, sm.full[slot][warp]);
        }
    };
    Place p = place_of<GRAD, S::TOK>(a, rank, ch);
    Pk<2> rate = rates(p);
    load(p, 0);
    int slot = 0;
    for (; rank < a.ranks; slot ^= 1) {
        next_place(a, rank, ch);
        const bool more = rank < a.ranks;
        const Place next = more ? place_of<GRAD, S::TOK>(a, rank, ch) : p;
        T *stage = (T *)(stages + slot * S::STAGE);
        if (TMA) {
            if (holds(p)) {
                if (asked && !wait_for(sm, sm.full[slot][warp], loaded[slot], a)) {
                    ok = false;
                    if (lane == 0)  // the copy may not land on the results, nor after the block
                        mbar_wait(smem_u32(&sm.full[slot][warp]), loaded[slot]);
                }
                loaded[slot] ^= 1;
            }
        } else {
            if constexpr (sizeof(T) == 4)
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
        }
        const int tok_end = ((GRAD ? a.ranks - 1 - p.rank : p.rank) + 1) * S::TOK;
        Pk<2> next_rate = rate;
        auto run = [&](auto mask) {
            LaneRun<T, GRAD, decltype(mask)::value, TMA> l{a, stage + 2 * lane, p, warp, lane, {}, {}};
            Pk<2> z, v;
            l.first(rate, z, v);
            const Pk<2> qw = GRAD ? decay(z) : one_minus_exp<2>(z);
            if (ok) {
                put2(&sm.q[slot][warp][2 * lane], qw);
                put2(&sm.v[slot][warp][2 * lane], v);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&sm.ready[slot]));
            if (more) {
                load(next, slot ^ 1);
                next_rate = rates(next);
            }
            Pk<2> h0 = pk_all<2>(0.0f);
            if (GRAD && a.h0 && l.token(S::L - 1) == 0) {
                float f[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int j = p.j0 + 2 * lane + k;
                    f[k] = j < a.dim ? a.h0[(long long)p.b * a.dim + j] : 0.0f;
                }
                h0 = pk<2>(f);
            }
            wait_for(sm, sm.ready[slot], phase, a);
            wait_for(sm, sm.entered[slot], phase, a);
            ok = ok && !stopped(sm);
            Pk<2> e = get2(&sm.enter[slot][2 * lane]);
            if (!ok)
                e = pk_all<2>(no_number());
            for (int w = 0; w < warp; ++w) {
                const Pk<2> m = get2(&sm.q[slot][w][2 * lane]);
                e = add_(GRAD ? kept(m, e) : fma_(neg_<2>(m), e, e), get2(&sm.v[slot][w][2 * lane]));
            }
            if constexpr (GRAD) {
                const Pk<2> sum = l.backward(e, rate, h0);
                put2(&sm.sums[warp][2 * lane], sum);
            } else {
                l.forward(e);
            }
        };
        if (!holds(p)) {
            LaneRun<T, GRAD, true, TMA> l{a, stage + 2 * lane, p, warp, lane, {}, {}};
            if (lane == 0)
                mbar_arrive(smem_u32(&sm.ready[slot]));
            if (more) {
                load(next, slot ^ 1);
                next_rate = rates(next);
            }
            wait_for(sm, sm.entered[slot], phase, a);
            ok = ok && !stopped(sm);
            if (TMA && lane == 0)
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int t = 0; t < S::L; ++t)
#pragma unroll
                for (int k = 0; k < S::OUT; ++k)
                    l.out(k, t, pk_all<2>(0.0f));
        } else if (tok_end <= p.n) {
            run(Flag<false>{});
        } else {
            run(Flag<true>{});
        }
        if (TMA) {
            fence_async_smem();
            __syncwarp();
            const int row0 = GRAD ? S::TOK - (warp + 1) * S::L : warp * S::L;
            if (lane == 0 && tok_end - S::TOK + row0 < a.time) {
#pragma unroll
                for (int k = 0; k < S::OUT; ++k)
                    tma_store(&maps.out[k], smem_u32(stage + (k * S::TOK + row0) * kChannels), p.j0,
                              tok_end - S::TOK + row0, p.b);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
        }
        phase ^= slot;
        p = next;
        rate = next_rate;
    }
    __syncwarp();
    if (GRAD && lane == 0)
        mbar_arrive(smem_u32(&sm.ready[slot]));
    if (TMA && lane == 0)
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

constexpr int kRateWarps = 8;

// drate = the tiles' sums: each warp of a block adds every eighth row, the block
// the warps'; 0 where the rate is not positive.
__global__ void __launch_bounds__(32 * kRateWarps) recur_rate_kernel(RecurArgs a)
{
    __shared__ float sm[kRateWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long j = (long long)blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (j < a.dim)
        for (long long row = warp; row < a.batch * a.ranks; row += kRateWarps)
            sum += a.part[row * a.dim + j];
    sm[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && j < a.dim) {
        for (int w = 1; w < kRateWarps; ++w)
            sum += sm[w][lane];
        a.drate[j] = a.rate[j] > 0.0f ? sum : 0.0f;
    }
}

// No token at all: the states pass through.
__global__ void recur_pass_kernel(const float *from, float *to, long long n)
{
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x)
        to[i] = from ? from[i] : 0.0f;
}

constexpr int kStepThreads = 128;

struct StepArgs {
    long long batch, dim, rows, state_stride, sx, sr, sh;
    float *state;
    const void *x, *r;
    const float *rate;
    const int32_t *slots;
    void *h;
};

// V neighbouring values as they lie in memory.
template <typename T, int V>
struct alignas(sizeof(T) * V) Row {
    T v[V];
};

// One token: V channels to a thread, a row of the batch to a row of blocks.
template <typename T, int V>
__global__ void __launch_bounds__(kStepThreads) recur_step_kernel(StepArgs a)
{
    const long long j = ((long long)blockIdx.x * kStepThreads + threadIdx.x) * V;
    if (j >= a.dim)
        return;
    const Row<float, V> rate = *reinterpret_cast<const Row<float, V> *>(a.rate + j);
    for (long long b = blockIdx.y; b < a.batch; b += gridDim.y) {
        const long long row = a.slots ? a.slots[b] : b;
        const bool in = row >= 0 && row < a.rows;
        Row<T, V> out;
        if (in) {
            const Row<T, V> x = *reinterpret_cast<const Row<T, V> *>((const T *)a.x + b * a.sx + j);
            const Row<T, V> r = *reinterpret_cast<const Row<T, V> *>((const T *)a.r + b * a.sr + j);
            Row<float, V> *at = reinterpret_cast<Row<float, V> *>(a.state + row * a.state_stride + j);
            Row<float, V> s = *at;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float lam = rate.v[k] < 0.0f ? 0.0f : rate.v[k];
                const float z = lam * sigma<1>(Pk<1>{to_f(r.v[k])}).v;
                s.v[k] = fmaf(one_minus_exp<1>(Pk<1>{z}).v, to_f(x.v[k]) - s.v[k], s.v[k]);
                out.v[k] = from_f<T>(s.v[k]);
            }
            *at = s;
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                out.v[k] = from_f<T>(0.0f);
        }
        *reinterpret_cast<Row<T, V> *>((T *)a.h + b * a.sh + j) = out;
    }
}

// Four channels to a thread where every row starts on the size of four.
template <typename T>
cudaError_t run_step(const StepArgs &a, cudaStream_t st)
{
    const size_t e = sizeof(T);
    const bool four = a.dim % 4 == 0 && a.state_stride % 4 == 0 && a.sx % 4 == 0 && a.sr % 4 == 0 && a.sh % 4 == 0 &&
                      !misaligned_to(a.state, 16) && !misaligned_to(a.rate, 16) && !misaligned_to(a.x, 4 * e) &&
                      !misaligned_to(a.r, 4 * e) && !misaligned_to(a.h, 4 * e);
    const long long per = kStepThreads * (four ? 4 : 1);
    const dim3 grid((unsigned)((a.dim + per - 1) / per), (unsigned)(a.batch < 65535 ? a.batch : 65535));
    if (four)
        recur_step_kernel<T, 4><<<grid, kStepThreads, 0, st>>>(a);
    else
        recur_step_kernel<T, 1><<<grid, kStepThreads, 0, st>>>(a);
    return cudaGetLastError();
}

bool takes(bstq_dtype d) { return d == BSTQ_F32 || d == BSTQ_BF16 || d == BSTQ_F16; }
size_t elem_of(bstq_dtype d) { return d == BSTQ_F32 ? 4 : 2; }

// Sizes up to 2^30 along each axis, 2^30 tiles of channels and 2^40 elements in
// all: offsets are held in 64 bits, tokens and tiles in 32.
bool sizes_ok(int64_t v) { return v >= 0 && v <= (1LL << 30); }
bool all_ok(int64_t batch, int64_t time, int64_t dim)
{
    return (double)batch * (double)time * (double)dim <= (double)(1LL << 40) &&
           (double)batch * ((double)dim / kChannels + 1.0) <= (double)(1LL << 30);
}

Seq seq_of(const int64_t *strides, int k, int64_t time, int64_t dim)
{
    if (strides)
        return Seq{strides[2 * k], strides[2 * k + 1]};
    return Seq{(long long)time * dim, (long long)dim};
}

bool strides_ok(const int64_t *strides, int count)
{
    if (strides)
        for (int i = 0; i < count; ++i)
            if (strides[i] < 0 || strides[i] > (1LL << 42))
                return false;
    return true;
}

bool apart(const Seq &s, int64_t batch, int64_t time, int64_t dim) { return rows_apart(dim, time, s.st, batch, s.sb); }

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

struct RecurPlan {
    long long ranks, cols, chains;
    size_t maps, part, total;  // offsets; the first 256 bytes hold the status
};
RecurPlan recur_plan(bstq_dtype dtype, int64_t batch, int64_t time, int64_t dim, bool grad)
{
    RecurPlan p;
    const int64_t tok = dtype == BSTQ_F32 ? (grad ? Tile<float, true>::TOK : Tile<float, false>::TOK)
                                          : (grad ? Tile<__half, true>::TOK : Tile<__half, false>::TOK);
    p.ranks = (time + tok - 1) / tok;
    p.cols = (dim + kChannels - 1) / kChannels;
    p.chains = batch * p.cols;
    p.maps = 256;
    p.part = p.maps + (p.ranks > 1 ? 8 * size_t(p.chains) * (p.ranks + (p.ranks + 3) / 4 + (p.ranks + 1) / 2) * kChannels
                                       : 0);  // maps, maps of four tiles, states
    p.total = p.part + (grad ? round256(4 * size_t(batch) * p.ranks * dim) : 0);
    return p;
}

// The SMs that the stream's context may use: a green context has a part of the
// device's, and blocks that wait for each other have to fit there.
int sms_of(cudaStream_t st, int device)
{
    typedef CUresult (*GetCtx)(CUstream, CUcontext *, CUgreenCtx *);
    typedef CUresult (*OfCtx)(CUcontext, CUdevResource *, CUdevResourceType);
    typedef CUresult (*OfGreen)(CUgreenCtx, CUdevResource *, CUdevResourceType);
    static const auto entry = [](const char *name) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult got;
        if (cudaGetDriverEntryPointByVersion(name, &f, 12050, cudaEnableDefault, &got) != cudaSuccess ||
            got != cudaDriverEntryPointSuccess)
            f = nullptr;
        return f;
    };
    static const GetCtx get = (GetCtx)entry("cuStreamGetCtx");
    static const OfCtx of_ctx = (OfCtx)entry("cuCtxGetDevResource");
    static const OfGreen of_green = (OfGreen)entry("cuGreenCtxGetDevResource");
    CUcontext ctx = nullptr;
    CUgreenCtx green = nullptr;
    CUdevResource r{};
    if (!get || !of_ctx || !of_green || get(st, &ctx, &green) != CUDA_SUCCESS ||
        (green ? of_green(green, &r, CU_DEV_RESOURCE_TYPE_SM) : of_ctx(ctx, &r, CU_DEV_RESOURCE_TYPE_SM)) != CUDA_SUCCESS)
        return device;
    const int sms = (int)r.sm.smCount;
    return sms > 0 && sms < device ? sms : device;
}

// Map of a batch x time x dim tensor in boxes of 64 channels by `rows` tokens.
// False where its rows do not start on 16 bytes: those go by ordinary loads.
bool tile_map(CUtensorMap *map, bstq_dtype dtype, const void *at, const Seq &s, const RecurArgs &a, int rows)
{
    const size_t e = elem_of(dtype);
    const long long st = a.time > 1 ? s.st : (a.dim + 7) & ~7LL;
    const long long sb = a.batch > 1 ? s.sb : st;
    if (misaligned_to(at, 16) || (st * e) % 16 || (sb * e) % 16 || st <= 0 || sb <= 0 || st * e >= (1ull << 40) ||
        sb * e >= (1ull << 40))
        return false;
    const CUtensorMapDataType type = dtype == BSTQ_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == BSTQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t dims[3] = {(cuuint64_t)a.dim, (cuuint64_t)a.time, (cuuint64_t)a.batch};
    const cuuint64_t strides[2] = {(cuuint64_t)(st * e), (cuuint64_t)(sb * e)};
    const cuuint32_t box[3] = {kChannels, (cuuint32_t)rows, 1}, unit[3] = {1, 1, 1};
    const EncodeFn fn = encode_fn();
    return fn && fn(map, type, 3, const_cast<void *>(at), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool GRAD>
cudaError_t run_tiles(bstq_dtype dtype, RecurArgs a, const RecurPlan &p, char *work, int sms, cudaStream_t st)
{
    using S = Tile<T, GRAD>;
    a.ranks = (int)p.ranks, a.cols = (int)p.cols, a.chains = (int)p.chains;
    a.status = (int *)work;
    a.wait = wait_limit();
    a.maps = (unsigned long long *)(work + p.maps);
    a.part = (float *)(work + p.part);
    RecurMaps maps;
    bool tma = tile_map(&maps.in[0], dtype, a.x, a.sx, a, S::L) && tile_map(&maps.in[1], dtype, a.r, a.sr, a, S::L);
    if (GRAD)
        tma = tma && tile_map(&maps.in[2], dtype, a.h_in, a.sh, a, S::L) &&
              tile_map(&maps.in[3], dtype, a.dh, a.sdh, a, S::L) &&
              tile_map(&maps.out[0], dtype, a.dx, a.sdx, a, S::L) &&
              tile_map(&maps.out[1], dtype, a.dr, a.sdr, a, S::L);
    else
        tma = tma && tile_map(&maps.out[0], dtype, a.h, a.sh, a, S::L);
    auto *kernel = tma ? recur_kernel<T, GRAD, true> : recur_kernel<T, GRAD, false>;
    // asked once for each device; every call finds the same
    static std::atomic<int> blocks[2][64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    int per_sm = dev < 64 ? blocks[tma][dev].load(std::memory_order_relaxed) : 0;
    if (per_sm == 0) {
        if ((err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, tile_smem<T, GRAD>())) !=
                cudaSuccess ||
            (err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, S::THREADS, tile_smem<T, GRAD>())) != cudaSuccess)
            return err;
        if (dev < 64)
            blocks[tma][dev].store(per_sm, std::memory_order_relaxed);
    }
    const long long tiles = p.ranks * p.chains, room = (long long)per_sm * (p.ranks > 1 ? sms_of(st, sms) : sms);
    const unsigned grid = (unsigned)(tiles < room ? tiles : room);
    a.group = a.chains >= (long long)grid ? 1 : kMaxGroup;
    // groups of one have no maps
    const size_t maps_bytes = a.group == 1 ? 0 : 8 * size_t(p.chains) * (p.ranks + (p.ranks + 3) / 4) * kChannels;
    const size_t states_bytes = 4 * size_t(p.chains) * ((p.ranks + a.group - 1) / a.group) * kChannels;
    a.states = (unsigned long long *)(work + p.maps + maps_bytes);
    a.step_rank = (int)(grid / a.chains), a.step_chain = (int)(grid % a.chains);
    if (a.ranks == 1) {  // no tile waits for another
        kernel<<<grid, S::THREADS, tile_smem<T, GRAD>(), st>>>(a, maps);
        return cudaGetLastError();
    }
    if ((err = cudaMemsetAsync(work + p.maps, 0xff, maps_bytes + states_bytes, st)) != cudaSuccess)
        return err;
    void *args[] = {&a, &maps};
    return cudaLaunchCooperativeKernel((const void *)kernel, dim3(grid), dim3(S::THREADS), args, tile_smem<T, GRAD>(), st);
}

cudaError_t pass_states(const float *from, float *to, long long n, cudaStream_t st)
{
    if (!to)
        return cudaSuccess;
    recur_pass_kernel<<<(unsigned)(n / 256 + 1 < 1024 ? n / 256 + 1 : 1024), 256, 0, st>>>(from, to, n);
    return cudaGetLastError();
}

}  // namespace
}  // namespace bstq

using namespace bstq;

extern "C" size_t bstq_recur_work_size(bstq_dtype dtype, int64_t batch, int64_t time, int64_t dim)
{
    if (!takes(dtype) || !sizes_ok(batch) || !sizes_ok(time) || !sizes_ok(dim) || !all_ok(batch, time, dim))
        return 0;
    return recur_plan(dtype, batch, time, dim, false).total;
}

extern "C" int bstq_recur(bstq_dtype dtype, int64_t batch, int64_t time, int64_t dim, const void *x, const void *r,
                          const float *rate, const float *h0, const int32_t *lengths, void *h, float *hT,
                          const int64_t *strides, void *work, void *stream)
{
    if (!takes(dtype))
        return -1;
    if (!sizes_ok(batch))
        return -2;
    if (!sizes_ok(time))
        return -3;
    if (!sizes_ok(dim) || !all_ok(batch, time, dim))
        return -4;
    if (batch == 0 || dim == 0)
        return 0;
    const size_t e = elem_of(dtype);
    if (time && (!x || misaligned_to(x, e)))
        return -5;
    if (time && (!r || misaligned_to(r, e)))
        return -6;
    if (!rate || misaligned_to(rate, 4))
        return -7;
    if (misaligned_to(h0, 4))
        return -8;
    if (misaligned_to(lengths, 4))
        return -9;
    if (time && (!h || misaligned_to(h, e)))
        return -10;
    if (misaligned_to(hT, 4))
        return -11;
    if (!strides_ok(strides, 6))
        return -12;
    if (!work || misaligned_to(work, 256))
        return -13;
    if (!apart(seq_of(strides, 2, time, dim), batch, time, dim))
        return -12;
    DevInfo di;
    if (!dev_info(di))
        return BSTQ_ERR_NODEVICE;
    RecurArgs a{};
    a.batch = batch, a.time = time, a.dim = dim;
    a.x = x, a.r = r, a.rate = rate, a.h0 = h0, a.lengths = lengths, a.h = h, a.hT = hT;
    a.sx = seq_of(strides, 0, time, dim), a.sr = seq_of(strides, 1, time, dim), a.sh = seq_of(strides, 2, time, dim);
    cudaStream_t st = (cudaStream_t)stream;
    const RecurPlan p = recur_plan(dtype, batch, time, dim, false);
    cudaError_t err;
    if (time == 0)
        err = pass_states(h0, hT, batch * dim, st);
    else if (dtype == BSTQ_F32)
        err = run_tiles<float, false>(dtype, a, p, (char *)work, di.sms, st);
    else if (dtype == BSTQ_BF16)
        err = run_tiles<__nv_bfloat16, false>(dtype, a, p, (char *)work, di.sms, st);
    else
        err = run_tiles<__half, false>(dtype, a, p, (char *)work, di.sms, st);
    return err == cudaSuccess ? 0 : cuda_fail(err, "gated recurrence");
}

extern "C" size_t bstq_recur_grad_work_size(bstq_dtype dtype, int64_t batch, int64_t time, int64_t dim)
{
    if (!bstq_recur_work_size(dtype, batch, time, dim))
        return 0;
    return recur_plan(dtype, batch, time, dim, true).total;
}

extern "C" int bstq_recur_grad(bstq_dtype dtype, int64_t batch, int64_t time, int64_t dim, const void *x,
                               const void *r, const float *rate, const void *h, const void *dh, const float *dhT,
                               const float *h0, const int32_t *lengths, void *dx, void *dr, float *drate, float *dh0,
                               const int64_t *strides, void *work, void *stream)
{
    if (!takes(dtype))
        return -1;
    if (!sizes_ok(batch))
        return -2;
    if (!sizes_ok(time))
        return -3;
    if (!sizes_ok(dim) || !all_ok(batch, time, dim))
        return -4;
    if (dim == 0)
        return 0;
    const size_t e = elem_of(dtype);
    const bool some = batch && time;
    if (some && (!x || misaligned_to(x, e)))
        return -5;
    if (some && (!r || misaligned_to(r, e)))
        return -6;
    if (!rate || misaligned_to(rate, 4))
        return -7;
    if (some && (!h || misaligned_to(h, e)))
        return -8;
    if (some && (!dh || misaligned_to(dh, e)))
        return -9;
    if (misaligned_to(dhT, 4))
        return -10;
    if (misaligned_to(h0, 4))
        return -11;
    if (misaligned_to(lengths, 4))
        return -12;
    if (some && (!dx || misaligned_to(dx, e)))
        return -13;
    if (some && (!dr || misaligned_to(dr, e)))
        return -14;
    if (!drate || misaligned_to(drate, 4))
        return -15;
    if (misaligned_to(dh0, 4))
        return -16;
    if (!strides_ok(strides, 12))
        return -17;
    if (!work || misaligned_to(work, 256))
        return -18;
    if (!apart(seq_of(strides, 4, time, dim), batch, time, dim) ||
        !apart(seq_of(strides, 5, time, dim), batch, time, dim))
        return -17;
    DevInfo di;
    if (!dev_info(di))
        return BSTQ_ERR_NODEVICE;
    RecurArgs a{};
    a.batch = batch, a.time = time, a.dim = dim;
    a.x = x, a.r = r, a.rate = rate, a.h_in = h, a.dh = dh, a.dhT = dhT, a.h0 = h0, a.lengths = lengths;
    a.dx = dx, a.dr = dr, a.drate = drate, a.dh0 = dh0;
    a.sx = seq_of(strides, 0, time, dim), a.sr = seq_of(strides, 1, time, dim), a.sh = seq_of(strides, 2, time, dim);
    a.sdh = seq_of(strides, 3, time, dim), a.sdx = seq_of(strides, 4, time, dim);
    a.sdr = seq_of(strides, 5, time, dim);
    cudaStream_t st = (cudaStream_t)stream;
    const RecurPlan p = recur_plan(dtype, batch, time, dim, true);
    cudaError_t err = cudaSuccess;
    if (!some)
        err = batch ? pass_states(dhT, dh0, batch * dim, st) : cudaSuccess;
    else if (dtype == BSTQ_F32)
        err = run_tiles<float, true>(dtype, a, p, (char *)work, di.sms, st);
    else if (dtype == BSTQ_BF16)
        err = run_tiles<__nv_bfloat16, true>(dtype, a, p, (char *)work, di.sms, st);
    else
        err = run_tiles<__half, true>(dtype, a, p, (char *)work, di.sms, st);
    if (err == cudaSuccess) {
        a.ranks = (int)p.ranks, a.part = (float *)((char *)work + p.part);
        recur_rate_kernel<<<(unsigned)((dim + 31) / 32), 32 * kRateWarps, 0, st>>>(a);
        err = cudaGetLastError();
    }
    return err == cudaSuccess ? 0 : cuda_fail(err, "gated recurrence, gradients");
}

extern "C" int bstq_recur_step(bstq_dtype dtype, int64_t batch, int64_t dim, int64_t rows, float *state,
                               int64_t state_stride, const void *x, const void *r, const float *rate,
                               const int32_t *slots, void *h, const int64_t *strides, void *stream)
{
    if (!takes(dtype))
        return -1;
    if (!sizes_ok(batch))
        return -2;
    if (!sizes_ok(dim) || !all_ok(batch, 1, dim))
        return -3;
    if (!sizes_ok(rows) || (!slots && rows < batch))
        return -4;
    if (batch == 0 || dim == 0)
        return 0;
    const size_t e = elem_of(dtype);
    if ((rows && !state) || misaligned_to(state, 4))
        return -5;
    if (state_stride < dim || state_stride > (1LL << 42))
        return -6;
    if (!x || misaligned_to(x, e))
        return -7;
    if (!r || misaligned_to(r, e))
        return -8;
    if (!rate || misaligned_to(rate, 4))
        return -9;
    if (misaligned_to(slots, 4))
        return -10;
    if (!h || misaligned_to(h, e))
        return -11;
    if (!strides_ok(strides, 3) || (strides && batch > 1 && strides[2] < dim))
        return -12;
    DevInfo di;
    if (!dev_info(di))
        return BSTQ_ERR_NODEVICE;
    StepArgs a{};
    a.batch = batch, a.dim = dim, a.rows = rows, a.state = state, a.state_stride = state_stride;
    a.x = x, a.r = r, a.rate = rate, a.slots = slots, a.h = h;
    a.sx = strides ? strides[0] : dim, a.sr = strides ? strides[1] : dim, a.sh = strides ? strides[2] : dim;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t err = dtype == BSTQ_F32    ? run_step<float>(a, st)
                            : dtype == BSTQ_BF16 ? run_step<__nv_bfloat16>(a, st)
                                                 : run_step<__half>(a, st);
    return err == cudaSuccess ? 0 : cuda_fail(err, "gated recurrence, one token");
}
