// sscan_gated.cu -- the gated linear recurrence with one state per channel,
//   r = sigmoid(a_raw + a_bias),  i = sigmoid(i_raw + i_bias),  s = rate softplus(Lam) r,
//   a = exp(-s),  m = sqrt(1 - a^2),   h_t = a_t h_{t-1} + m_t i_t u_t,   out_t = h_t,
// for every (batch, channel); its backward pass and its one-token step.
//
// One pass over the sequence.  A block owns a tile of kWarps x S steps by 32 V channels (S = 16
// forward, 8 backward): each of its kWarps working warps scans S consecutive steps from zero
// with the gates' results in registers, the warps' affine maps h -> A h + H are combined through
// shared memory, the state entering the tile comes from the tiles before it, and a second sweep
// over the registers writes the outputs.  So every input is read once and every output written
// once, however the sequence is split.
//
// A fixed number of blocks take tile after tile.  While a tile is computed, the next one's inputs
// are on their way to shared memory.  Results overwrite the inputs they came from there.  Rows and widths on 16-byte boundaries travel by
// TMA, which also fills and clips the edges; others by the working warps.
//
// The carry between tiles: tickets run in time order, so whatever a tile waits for is held by a
// block that has started and waits only for earlier tiles.  One extra warp of a block (carry_in)
// waits for the earlier tiles' maps while the others compute; another (carry_out) publishes this
// tile's map as soon as it is known.  Tiles are composed in a fixed tree: the maps of kFan tiles
// make a group's, published by its last tile, and the state entering kFan groups is handed on by
// their last tile.  So two runs round alike, a tile reads at most 2 (kFan - 1) maps and one state,
// all at once, and the serial chain has one hop per kFan^2 tiles.  A published word is its own
// flag: the arrays start as all ones, a NaN that no arithmetic returns, and each 8-byte word is
// stored and polled whole, so no fence or second round trip is needed.
//
// 8 x 2048 x 5120 bf16 forward: 126 us, 5.3 TB/s (82% of the measured copy bandwidth), issue slots
// 63% busy; 8 x 2048 x 1536: forward and backward 139 us, a third and two thirds; 131072 x 1536: 573 us, there the
// tiles of a column that run at the same time wait for each other's maps.
//
// Per element the forward moves 4 I/O elements against 4 special-function operations (5 where a
// channel's decay can pass exp(-1/4)) and 34 issued instructions; two elements, V = 2
// channels or two steps, share each packed fp32 instruction.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <type_traits>

#include "sscan_check.cuh"
#include "sscan_host.h"
#include "sscan_launch.h"
#include "sscan_math.cuh"
#include "sscan_plan.h"
#include "sscan_rowsum.cuh"
#include "sscan_tma.cuh"
#include "sscan_vec.cuh"

namespace sscan {

__device__ unsigned int g_device_error_gated = 0;

namespace {

constexpr int kWarps = 8;
constexpr int kStepsFwd = 16, kStepsBwd = 8; // steps per warp
constexpr int kCkpt = kWarps * kStepsBwd;    // checkpoint interval: a tile of the backward
constexpr int kFan = 8;                      // tiles per group, groups per hop of the serial chain
constexpr int kThreads = 32 * (kWarps + 2);  // the working warps, carry_in's and carry_out's
constexpr uint32_t kPollLimit = 1u << 20;
constexpr unsigned long long kUnset = ~0ull;

// Every array starts as all ones.
struct Chain {
    unsigned int* ticket;         // null: one tile per sequence, no carry
    unsigned long long* maps;     // [cols][tiles][32 V] (A, H) of a tile
    unsigned long long* groups;   // [cols][ngroups][32 V] (A, H) of kFan tiles
    unsigned long long* states;   // [cols][nsupers][32 V] (h, 0): the state entering kFan groups
    int64_t tiles, ngroups, nsupers, cols;
};

struct GatedArgs {
    int64_t batch, L, D, nblk;  // nblk: channel blocks of 32 V
    const void *u, *a_raw, *i_raw;
    const float *Lam, *a_bias, *i_bias, *h0;
    float rate;
    void* out;       // (batch, L, D) or null (checkpoints only)
    float* h_last;   // (batch, D) or null
    float* ckpt;     // (batch, ceil(L / kCkpt), D) or null: the state before every kCkpt-th step
    Chain chain;
    // backward
    const void* dout;
    const float* ckpt_in;
    void *du, *da_raw, *di_raw;
    float* dh0;      // (batch, D) or null
    float* part;     // [batch * tiles][3][D]: sums of ds r, da_raw, di_raw over the tile
    // step
    float* state;    // (batch, D)
};

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

__device__ __forceinline__ float rsqrt_fast(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / sqrt(om), and a large finite value where om has underflowed to 0 (its products with om and
// with s are then 0): 1.2e-38 is the least that the reciprocal root does not take for 0
__device__ __forceinline__ float2 rsqrt2(float2 om) {
    return make_float2(rsqrt_fast(fmaxf(om.x, 1.2e-38f)), rsqrt_fast(fmaxf(om.y, 1.2e-38f)));
}

// a = exp(-s) and om = 1 - a^2 = e (2 - e), with e = 1 - a.  For s < 1/4, e comes from its Taylor
// series to s^6 (the dropped s^7/5040 is below 5.5e-8 of e, the same size as e's rounding): the difference
// 1 - a would cancel, and a long memory multiplies a's error by its length.  From 1/4 on (kAny: some s may
// be there) a is the exponential itself, which keeps its relative precision however small it is (1 - e
// would round it to a multiple of 2^-24, and every gradient through the state is a multiple of a).
template <bool kAny>
__device__ __forceinline__ void decay2(float2 s, float2& a, float2& om) {
    float2 p = fma2(s, splat(-1.f / 720.f), splat(1.f / 120.f));
    p = fma2(s, p, splat(-1.f / 24.f));
    p = fma2(s, p, splat(1.f / 6.f));
    p = fma2(s, p, splat(-0.5f));
    p = fma2(s, p, splat(1.f));
    float2 e = mul2(s, p);
    a = fma2(e, splat(-1.f), splat(1.f));
    if (kAny) {
        if (!(s.x < 0.25f)) a.x = ex2(-s.x * kLog2e), e.x = 1.f - a.x;
        if (!(s.y < 0.25f)) a.y = ex2(-s.y * kLog2e), e.y = 1.f - a.y;
    }
    om = mul2(e, fma2(e, splat(-1.f), splat(2.f)));
}

// min(x, 127) that keeps a NaN
__device__ __forceinline__ float min_nan(float x) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(127.f));
    return y;
}

// a b, with results below 2^-126 as 0
__device__ __forceinline__ float2 mul2_ftz(float2 a, float2 b) {
    float2 y;
    asm("{\n\t.reg .b64 a, b, y;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.ftz.f32x2 y, a, b;\n\t"
        "mov.b64 {%0, %1}, y;\n\t}"
        : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return y;
}

// sigmoid(x + bias) of both gates for two elements: 1 / D with D = 1 + 2^q, q = nbias - log2(e) x, nbias =
// -log2(e) bias.  Both come from one reciprocal, 1 / D_r = D_i / (D_r D_i), with D_i scaled by 2^-100, so that the
// product is in fp32's range while one gate is open.  (The exponent itself is not shifted: its rounding would be that
// of a number near 100.)  A gate goes down to 2^-126, then to 0: from q = 127 on, where q is held, and for an x
// of -inf, it is exactly that, and the other gate is as it would be.  Both are 0 where their product is below 2^-226.
__device__ __forceinline__ void gates2(float2 xr, float2 xi, float2 nbr, float2 nbi, float2& r, float2& i) {
    const float2 qr = fma2(xr, splat(-kLog2e), nbr), qi = fma2(xi, splat(-kLog2e), nbi), scale = splat(0x1p-100f);
    const float2 er = make_float2(ex2(min_nan(qr.x)), ex2(min_nan(qr.y)));
    const float2 ei = make_float2(ex2(min_nan(qi.x)), ex2(min_nan(qi.y)));
    const float2 dr = add2(er, splat(1.f)), di = fma2(ei, scale, scale), p = mul2(dr, di);
    const float2 rp = make_float2(rcp(p.x), rcp(p.y));
    r = mul2_ftz(di, rp);
    i = mul2_ftz(mul2(dr, scale), rp);
}

// rate * softplus(Lam), once per channel of a block
__device__ __forceinline__ float decay_rate(float lam, float rate) {
    return rate * (lam > 20.f ? lam : log1pf(expf(lam)));
}

// A published word, read and written whole past the L1.
__device__ __forceinline__ unsigned long long poll_word(const unsigned long long* p) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void put_word(unsigned long long* p, float a, float h) {
    const unsigned long long v = ((unsigned long long)__float_as_uint(h) << 32) | __float_as_uint(a);
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}

// Composes the n <= kFan - 1 maps of V channels per lane that start at words + first, each `V * 32`
// words after the one before, onto (A, H); false when one did not come in time.
template <int V>
__device__ __forceinline__ bool take_maps(const unsigned long long* words, int64_t first, int64_t extent, int n,
                                          float (&A)[V], float (&H)[V], uint32_t limit) {
    // a map that is not asked for is the identity (1, 0)
    unsigned long long m[kFan - 1][V];
    const unsigned long long* p = words + first;
    bool ready = false;
#pragma unroll 1
    for (uint32_t tries = 0; tries < limit && !ready; ++tries) {
        ready = true;
#pragma unroll
        for (int i = 0; i < kFan - 1; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v)
                m[i][v] = i < n && in_range(first + i * 32 * V + v, extent) ? poll_word(p + i * 32 * V + v) : 0x3f800000ull;
#pragma unroll
        for (int i = 0; i < kFan - 1; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) ready = ready && m[i][v] != kUnset;
    }
#pragma unroll
    for (int i = 0; i < kFan - 1; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float a = __uint_as_float((unsigned int)m[i][v]), h = __uint_as_float((unsigned int)(m[i][v] >> 32));
            H[v] = fmaf(a, H[v], h);
            A[v] *= a;
        }
    return ready;
}

// What a block knows of the tile it works on.
struct TileId {
    unsigned int k;      // rank in chain order
    unsigned int col, b, blk;
};

struct ChainSmem {
    TileId tile[4];          // by iteration
    int gave_up;             // a wait for a copy ran out: this block starts no more
    float rate[2][64];       // rate softplus(Lam) of the tile's channels, by iteration
    float in[64];            // the state entering the tile
    float2 group[64];        // composed maps of the group's earlier tiles
};

// A copy has not come in time.  The block takes no tile after the one that it has drawn (a barrier's phase may be
// incomplete), and tiles that wait for what it does not do give up in their turn.
__device__ __forceinline__ void give_up(ChainSmem& s, unsigned int err) {
    *reinterpret_cast<volatile int*>(&s.gave_up) = 1;
    atomicOr(&g_device_error_gated, err);
}

// Barriers of a block besides 0: 1 the tile's maps are in shared memory (working warps and
// carry_out's), 2 the entering state is (all warps), 3 the group's earlier tiles are composed
// (the two carry warps), 4 the working warps alone.
__device__ __forceinline__ void sync_maps() { asm volatile("bar.sync 1, %0;" ::"n"(32 * (kWarps + 1)) : "memory"); }
__device__ __forceinline__ void sync_state() { asm volatile("bar.sync 2, %0;" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ void sync_work() { asm volatile("bar.sync 4, %0;" ::"n"(32 * kWarps) : "memory"); }
__device__ __forceinline__ void sync_group() { asm volatile("bar.sync 3, 64;" ::: "memory"); }

__device__ __forceinline__ bool closes_group(unsigned int k) { return k % kFan == kFan - 1; }
__device__ __forceinline__ bool closes_super(unsigned int k) { return k % (kFan * kFan) == kFan * kFan - 1; }

// carry_in's warp: the state entering tile t of the chain, into s.in; `first` enters tile 0.  A
// wait that gives up raises `err` and goes on with what it has, and so do the tiles after it.
template <int V>
__device__ __forceinline__ void carry_in(const Chain& c, const TileId& t, const float (&first)[V], float (&state)[V],
                                         ChainSmem& s, unsigned int err, uint32_t limit = kPollLimit) {
    const int lane = threadIdx.x & 31;
    const int64_t k = t.k, g = k / kFan, sp = g / kFan, W = 32 * V;
    float A[V], H[V], Ag[V], Hg[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = Ag[v] = 1.f, H[v] = Hg[v] = 0.f, state[v] = first[v];
    const int64_t lv = lane * V;
    bool ok = take_maps<V>(c.maps, (t.col * c.tiles + g * kFan) * W + lv, c.cols * c.tiles * W, (int)(k - g * kFan), A, H, limit);
    if (closes_group(t.k)) {
#pragma unroll
        for (int v = 0; v < V; ++v) s.group[lv + v] = make_float2(A[v], H[v]);
        sync_group();
    }
    ok = take_maps<V>(c.groups, (t.col * c.ngroups + sp * kFan) * W + lv, c.cols * c.ngroups * W, (int)(g - sp * kFan), Ag, Hg, limit) && ok;
    if (sp > 0) {
        const int64_t at = (t.col * c.nsupers + sp) * W + lv;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            unsigned long long m = kUnset;
            for (uint32_t tries = 0; tries < limit && m == kUnset; ++tries) {
                if (tries) __nanosleep(32);
                m = in_range(at + v, c.cols * c.nsupers * W) ? poll_word(c.states + at + v) : 0ull;
            }
            ok = ok && m != kUnset;
            state[v] = __uint_as_float((unsigned int)m);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        state[v] = fmaf(A[v], fmaf(Ag[v], state[v], Hg[v]), H[v]);
        s.in[lv + v] = state[v];
    }
    if (!ok) atomicOr(&g_device_error_gated, err);
}

// carry_out's warp, once the tile's own map (A, H) is known: publishes it, or the group's.
template <int V>
__device__ __forceinline__ void publish_map(const Chain& c, const TileId& t, const float (&A)[V], const float (&H)[V],
                                            const ChainSmem& s) {
    const int lane = threadIdx.x & 31;
    const int64_t W = 32 * V, lv = lane * V, k = t.k, g = k / kFan;
    if (closes_group(t.k)) {
        sync_group();
        if (k + 1 >= c.tiles || closes_super(t.k)) return;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float2 m = s.group[lv + v];
            const int64_t at = (t.col * c.ngroups + g) * W + lv + v;
            if (in_range(at, c.cols * c.ngroups * W)) put_word(c.groups + at, A[v] * m.x, fmaf(A[v], m.y, H[v]));
        }
    } else if (k + 1 < c.tiles) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t at = (t.col * c.tiles + k) * W + lv + v;
            if (in_range(at, c.cols * c.tiles * W)) put_word(c.maps + at, A[v], H[v]);
        }
    }
}

// And once the entering state is: the state after the tile, for the next kFan groups.
template <int V>
__device__ __forceinline__ void publish_state(const Chain& c, const TileId& t, const float (&after)[V]) {
    const int64_t W = 32 * V, lv = (threadIdx.x & 31) * V, k = t.k, at = (t.col * c.nsupers + k / (kFan * kFan) + 1) * W + lv;
    if (!closes_super(t.k) || k + 1 >= c.tiles) return;
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (in_range(at + v, c.cols * c.nsupers * W)) put_word(c.states + at + v, after[v], 0.f);
}

// The next ticket of this block, as a tile (k >= tiles: none left).  One thread.
__device__ __forceinline__ TileId draw_tile(const GatedArgs& g, unsigned int iteration) {
    const unsigned int place = g.chain.ticket ? atomicAdd(g.chain.ticket, 1u) + 1u : blockIdx.x + iteration * gridDim.x;
    const unsigned int cols = (unsigned int)g.chain.cols, k = place / cols, col = place - k * cols;
    const unsigned int nblk = (unsigned int)g.nblk, b = col / nblk;
    return TileId{k, col, b, col - b * nblk};
}

// Rates of a tile's 32 V channels (one warp).
template <int V>
__device__ __forceinline__ void fill_rates(const GatedArgs& g, const TileId& t, float* rates) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t x = (int64_t)t.blk * 32 * V + v * 32 + lane;
        rates[v * 32 + lane] = x < g.D && in_range(x, g.D) ? decay_rate(__ldg(g.Lam + x), g.rate) : 0.f;
    }
}

// ROWS rows of 32 V elements of a (batch, L, D) tensor from (b, t0, d0) into shared memory, zeros
// outside, by the working warps.
template <typename T, int V, int ROWS>
__device__ __forceinline__ void fetch_rows(T* dst, const void* src, const GatedArgs& g, int64_t b, int64_t t0, int64_t d0) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const bool live = d0 + lane * V < g.D;
    const T* from = static_cast<const T*>(src) + (b * g.L + t0 + w) * g.D + d0 + lane * V;
#pragma unroll 8
    for (int r = w; r < ROWS; r += kWarps, from += kWarps * g.D) {
        Vec<T, V> v;
        v.zero();
        if (live && t0 + r < g.L) v.load(from);
        v.store(dst + (r * 32 + lane) * V);
    }
}

template <typename T, int V, int TENSORS, int STEPS>
struct GatedSmem {
    static constexpr int ROWS = kWarps * STEPS, TILE = ROWS * 32 * V, BYTES = TILE * (int)sizeof(T);
    alignas(128) T rows[2][TENSORS][TILE];  // by iteration
    uint64_t full[2];
    float2 AH[kWarps][32 * V];              // maps of the warps; then of all the warps before each
    ChainSmem c;
};

// Element pair k (V = 2: step k; V = 1: steps k and k + 1) of a thread's column of a tile.
template <typename T, int V>
__device__ __forceinline__ float2 pair_of(const T* rows, int k) {
    float x[V];
    load_shared<V>(rows + k * 32 * V, x);
    if constexpr (V == 2) {
        return make_float2(x[0], x[1]);
    } else {
        float y[V];
        load_shared<V>(rows + (k + 1) * 32 * V, y);
        return make_float2(x[0], y[0]);
    }
}

// Keeps the compiler from moving shared-memory loads across: left to itself it gathers those of
// all steps at the start and spills what is already computed (about 1 KB per thread).
__device__ __forceinline__ void hold_loads() { asm volatile("" ::: "memory"); }

// The gates and the recurrence's terms for the STEPS x V elements of a thread's column of a tile,
// two at a time: the V = 2 channels of a step, or two steps of the one channel.
template <typename T, int V, int STEPS, bool kAny, typename Out>
__device__ __forceinline__ void gate_terms(float2 c, float2 na, float2 ni, const T* ar, const T* ir, const T* u, Out out) {
#pragma unroll
    for (int k = 0; k < STEPS; k += 3 - V) {
        if (k % 4 == 0) hold_loads();
        float2 r, i, a, om;
        gates2(pair_of<T, V>(ar, k), pair_of<T, V>(ir, k), na, ni, r, i);
        decay2<kAny>(mul2(c, r), a, om);
        const float2 m = mul2(om, rsqrt2(om));
        out(k, a, mul2(mul2(m, i), pair_of<T, V>(u, k)), r, i);
    }
}

template <int V, int STEPS>
__device__ __forceinline__ void set_pair(float (&v)[STEPS][V], int k, float2 x) {
    v[k][0] = x.x;
    if constexpr (V == 2) v[k][1] = x.y;
    else v[k + 1][0] = x.y;
}

// Starts a tile's inputs on their way to buffer `buf`: one thread, by TMA.
template <int TENSORS, typename Smem>
__device__ __forceinline__ void tma_fetch(Smem& sm, int buf, int first, int n, const CUtensorMap* const (&maps)[TENSORS],
                                          const TileId& t, int row, int width) {
    const uint32_t bar = smem_u32(&sm.full[buf]);
    if (first == 0) mbar_expect_tx(bar, TENSORS * Smem::BYTES);
    for (int i = first; i < first + n; ++i)
        tma_load_3d(smem_u32(sm.rows[buf][i]), maps[i], (int)t.blk * width, row, (int)t.b, bar);
}

template <typename T, int V, bool kTma>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1)
    gated_fwd_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_i,
                     const __grid_constant__ CUtensorMap tm_u, const __grid_constant__ CUtensorMap tm_out, GatedArgs g) {
    constexpr int S = kStepsFwd;
    using Smem = GatedSmem<T, V, 3, S>;
    constexpr int ROWS = Smem::ROWS;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, lv = lane * V;
    const unsigned int tiles = (unsigned int)g.chain.tiles;
    const CUtensorMap* const maps[3] = {&tm_a, &tm_i, &tm_u};
    if (threadIdx.x == 0) {
        sm.c.tile[0] = draw_tile(g, 0);
        sm.c.gave_up = 0;
        if (kTma) {
            mbar_init(smem_u32(&sm.full[0]), 1);
            mbar_init(smem_u32(&sm.full[1]), 1);
            fence_proxy_async();
        }
    }
    __syncthreads();
    if (w == kWarps + 1 && sm.c.tile[0].k < tiles) {
        if (kTma && lane == 0) tma_fetch<3>(sm, 0, 0, 3, maps, sm.c.tile[0], (int)sm.c.tile[0].k * ROWS, 32 * V);
        fill_rates<V>(g, sm.c.tile[0], sm.c.rate[0]);
    }

    for (unsigned int it = 0;; ++it) {
        __syncthreads();  // this tile's place and rates are here, and the last tile is done with
        const TileId t = sm.c.tile[it & 3];
        const int buf = it & 1;
        if (w == kWarps + 1 && lane == 0) {
            // the last tile's outputs leave, then the next tile's inputs may take their place
            const bool stop = kTma && *reinterpret_cast<volatile int*>(&sm.c.gave_up);
            TileId next = t.k < tiles ? draw_tile(g, it + 1) : t;
            if (stop) next.k = tiles;
            sm.c.tile[(it + 1) & 3] = next;
            const bool more = kTma && next.k < tiles;
            if (kTma && it > 0 && g.out) {
                const TileId p = sm.c.tile[(it - 1) & 3];
                tma_store_3d(&tm_out, (int)p.blk * 32 * V, (int)p.k * ROWS, (int)p.b, smem_u32(sm.rows[buf ^ 1][2]));
            }
            if (more) tma_fetch<3>(sm, buf ^ 1, 0, 2, maps, next, (int)next.k * ROWS, 32 * V);
            if (kTma) tma_store_wait_read_0();
            if (more) tma_fetch<3>(sm, buf ^ 1, 2, 1, maps, next, (int)next.k * ROWS, 32 * V);
        }
        if (t.k >= tiles) break;
        const int64_t b = t.b, d = (int64_t)t.blk * 32 * V + lv;
        const bool live = d < g.D;  // V divides D, so a lane's channels are all inside or all outside
        if (w == kWarps) {
            float first[V], state[V];
#pragma unroll
            for (int v = 0; v < V; ++v) first[v] = live && g.h0 && in_range(b * g.D + d + v, g.batch * g.D) ? __ldg(g.h0 + b * g.D + d + v) : 0.f;
            carry_in<V>(g.chain, t, first, state, sm.c, 1u);
            sync_state();
            continue;
        }
        if (w == kWarps + 1) {
            __syncwarp();
            if (sm.c.tile[(it + 1) & 3].k < tiles) fill_rates<V>(g, sm.c.tile[(it + 1) & 3], sm.c.rate[buf ^ 1]);
            sync_maps();
            float A[V], H[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                A[v] = 1.f, H[v] = 0.f;
#pragma unroll
                for (int q = 0; q < kWarps; ++q) {
                    const float2 m = sm.AH[q][lv + v];
                    sm.AH[q][lv + v] = make_float2(A[v], H[v]);
                    H[v] = fmaf(m.x, H[v], m.y);
                    A[v] *= m.x;
                }
            }
            publish_map<V>(g.chain, t, A, H, sm.c);
            sync_state();
#pragma unroll
            for (int v = 0; v < V; ++v) H[v] = fmaf(A[v], sm.c.in[lv + v], H[v]);
            publish_state<V>(g.chain, t, H);
            if (live && g.h_last && t.k == tiles - 1) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (in_range(b * g.D + d + v, g.batch * g.D)) g.h_last[b * g.D + d + v] = H[v];
            }
            continue;
        }

        const int64_t t0 = (int64_t)t.k * ROWS + w * S;
        const int own = w * S * 32 * V + lv;
        T *ar = sm.rows[buf][0] + own, *ir = sm.rows[buf][1] + own, *u = sm.rows[buf][2] + own;
        if (kTma) {
            if (!mbar_wait(smem_u32(&sm.full[buf]), (it >> 1) & 1) && lane == 0) give_up(sm.c, 1u);
        } else {
            const int64_t r0 = (int64_t)t.k * ROWS, d0 = (int64_t)t.blk * 32 * V;
            fetch_rows<T, V, ROWS>(sm.rows[buf][0], g.a_raw, g, b, r0, d0);
            fetch_rows<T, V, ROWS>(sm.rows[buf][1], g.i_raw, g, b, r0, d0);
            fetch_rows<T, V, ROWS>(sm.rows[buf][2], g.u, g, b, r0, d0);
            sync_work();
        }
        float nab[V], nib[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            nab[v] = live && g.a_bias && in_range(d + v, g.D) ? -kLog2e * __ldg(g.a_bias + d + v) : 0.f;
            nib[v] = live && g.i_bias && in_range(d + v, g.D) ? -kLog2e * __ldg(g.i_bias + d + v) : 0.f;
        }
        const float2 c = make_float2(sm.c.rate[buf][lv], sm.c.rate[buf][lv + V - 1]);
        const float2 na = make_float2(nab[0], nab[V - 1]), ni = make_float2(nib[0], nib[V - 1]);
        float a[S][V], x[S][V];
        auto out = [&](int k, float2 pa, float2 px, float2, float2) {
            set_pair<V, S>(a, k, pa);
            set_pair<V, S>(x, k, px);
        };
        // r <= 1, so a rate below 1/4 keeps every s of the warp there
        if (__any_sync(0xffffffffu, !(c.x < 0.25f && c.y < 0.25f))) gate_terms<T, V, S, true>(c, na, ni, ar, ir, u, out);
        else gate_terms<T, V, S, false>(c, na, ni, ar, ir, u, out);
        if (t0 + S > g.L) {  // past the end: the identity map
#pragma unroll
            for (int k = 0; k < S; ++k)
                if (t0 + k >= g.L) {
#pragma unroll
                    for (int v = 0; v < V; ++v) a[k][v] = 1.f, x[k][v] = 0.f;
                }
        }
        float A[V], H[V];
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
        for (int k = 0; k < S; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                H[v] = fmaf(a[k][v], H[v], x[k][v]);
                A[v] *= a[k][v];
            }
#pragma unroll
        for (int v = 0; v < V; ++v) sm.AH[w][lv + v] = make_float2(A[v], H[v]);
        sync_maps();
        sync_state();
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float2 m = sm.AH[w][lv + v];
            h[v] = fmaf(m.x, sm.c.in[lv + v], m.y);
        }
        if (g.ckpt && t0 % kCkpt == 0 && t0 < g.L && live) {
            const int64_t rows = (g.L + kCkpt - 1) / kCkpt;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t at = (b * rows + t0 / kCkpt) * g.D + d + v;
                if (in_range(at, g.batch * rows * g.D)) g.ckpt[at] = h[v];
            }
        }
        if (!g.out) continue;
#pragma unroll
        for (int k = 0; k < S; ++k) {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fmaf(a[k][v], h[v], x[k][v]);
            if (kTma) store_vec<V>(u + k * 32 * V, h);
            else if (live && t0 + k < g.L) store_vec<V>(static_cast<T*>(g.out) + (b * g.L + t0 + k) * g.D + d, h);
        }
        if (kTma) fence_proxy_async();
    }
    if (kTma && w == kWarps + 1 && lane == 0) {
        tma_store_wait_all();
        // every copy has been waited for, or is now: shared memory is given up with nothing in flight on it
        if (*reinterpret_cast<volatile int*>(&sm.c.gave_up))
            for (int k = 0; k < 2; ++k) mbar_drain(smem_u32(&sm.full[k]));
    }
}

// The adjoint e_t that step t hands to h_{t-1} is affine in the one it gets: with
// g_t = dout_t + e_{t+1},  e_t = a_t g_t.  Tiles run from the last to the first; the state
// entering a tile is known (a checkpoint), so the forward states are rebuilt without a wait.
//   du = g m i,   di_raw = g m i u (1 - i),
//   ds = -e_t (h_{t-1} - (a / m) i u),   da_raw = ds s (1 - r),   dLam = sum ds r * rate sigmoid(Lam)
// Where s underflows to 0, m = 0 and its slope's limit is not finite; that term is left out.
template <typename T, int V>
struct GatedBwdSmem : GatedSmem<T, V, 4, kStepsBwd> {
    float2 AE[kWarps][32 * V];              // maps of the adjoint, as AH holds those of the state
    float red[3][kWarps][32 * V];
};

template <typename T, int V, bool kTma>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1)
    gated_bwd_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_i,
                     const __grid_constant__ CUtensorMap tm_u, const __grid_constant__ CUtensorMap tm_g,
                     const __grid_constant__ CUtensorMap tm_da, const __grid_constant__ CUtensorMap tm_di,
                     const __grid_constant__ CUtensorMap tm_du, GatedArgs g) {
    constexpr int S = kStepsBwd;
    using Smem = GatedBwdSmem<T, V>;
    constexpr int ROWS = Smem::ROWS;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, lv = lane * V;
    const unsigned int tiles = (unsigned int)g.chain.tiles;
    const CUtensorMap* const maps[4] = {&tm_g, &tm_a, &tm_i, &tm_u};
    auto row_of = [&](const TileId& t) { return (int)(tiles - 1 - t.k) * ROWS; };
    if (threadIdx.x == 0) {
        sm.c.tile[0] = draw_tile(g, 0);
        sm.c.gave_up = 0;
        if (kTma) {
            mbar_init(smem_u32(&sm.full[0]), 1);
            mbar_init(smem_u32(&sm.full[1]), 1);
            fence_proxy_async();
        }
    }
    __syncthreads();
    if (w == kWarps + 1 && sm.c.tile[0].k < tiles) {
        if (kTma && lane == 0) tma_fetch<4>(sm, 0, 0, 4, maps, sm.c.tile[0], row_of(sm.c.tile[0]), 32 * V);
        fill_rates<V>(g, sm.c.tile[0], sm.c.rate[0]);
    }

    for (unsigned int it = 0;; ++it) {
        __syncthreads();  // this tile's place and rates are here, and the last tile is done with but for its sums
        const TileId t = sm.c.tile[it & 3];
        const int buf = it & 1;
        if (w == kWarps + 1 && lane == 0) {
            const bool stop = kTma && *reinterpret_cast<volatile int*>(&sm.c.gave_up);
            TileId next = t.k < tiles ? draw_tile(g, it + 1) : t;
            if (stop) next.k = tiles;
            sm.c.tile[(it + 1) & 3] = next;
            const bool more = kTma && next.k < tiles;
            if (kTma && it > 0) {
                const TileId p = sm.c.tile[(it - 1) & 3];
                const int x = (int)p.blk * 32 * V, y = row_of(p);
                tma_store_3d_nocommit(&tm_da, x, y, (int)p.b, smem_u32(sm.rows[buf ^ 1][1]));
                tma_store_3d_nocommit(&tm_di, x, y, (int)p.b, smem_u32(sm.rows[buf ^ 1][2]));
                tma_store_3d_nocommit(&tm_du, x, y, (int)p.b, smem_u32(sm.rows[buf ^ 1][3]));
                tma_commit();
            }
            if (more) tma_fetch<4>(sm, buf ^ 1, 0, 1, maps, next, row_of(next), 32 * V);
            if (kTma) tma_store_wait_read_0();
            if (more) tma_fetch<4>(sm, buf ^ 1, 1, 3, maps, next, row_of(next), 32 * V);
        }
        if (it > 0 && w < 3) {
            // the last tile's sums over its warps
            const TileId p = sm.c.tile[(it - 1) & 3];
            const int64_t d = (int64_t)p.blk * 32 * V + lv, j = tiles - 1 - p.k;
            if (d < g.D) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float s = 0.f;
#pragma unroll
                    for (int q = 0; q < kWarps; ++q) s += sm.red[w][q][lv + v];
                    const int64_t at = (((int64_t)p.b * g.chain.tiles + j) * 3 + w) * g.D + d + v;
                    if (in_range(at, g.batch * g.chain.tiles * 3 * g.D)) g.part[at] = s;
                }
            }
        }
        if (t.k >= tiles) break;
        const int64_t b = t.b, j = tiles - 1 - t.k, d = (int64_t)t.blk * 32 * V + lv;
        const bool live = d < g.D;
        if (w == kWarps) {
            float zero[V], state[V];
#pragma unroll
            for (int v = 0; v < V; ++v) zero[v] = 0.f;
            carry_in<V>(g.chain, t, zero, state, sm.c, 2u);
            sync_state();
            continue;
        }
        if (w == kWarps + 1) {
            __syncwarp();
            if (sm.c.tile[(it + 1) & 3].k < tiles) fill_rates<V>(g, sm.c.tile[(it + 1) & 3], sm.c.rate[buf ^ 1]);
            sync_maps();
            float A[V], E[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                A[v] = 1.f, E[v] = 0.f;
#pragma unroll
                for (int q = kWarps - 1; q >= 0; --q) {
                    const float2 m = sm.AE[q][lv + v];
                    sm.AE[q][lv + v] = make_float2(A[v], E[v]);
                    E[v] = fmaf(m.x, E[v], m.y);
                    A[v] *= m.x;
                }
            }
            publish_map<V>(g.chain, t, A, E, sm.c);
            sync_state();
#pragma unroll
            for (int v = 0; v < V; ++v) E[v] = fmaf(A[v], sm.c.in[lv + v], E[v]);
            publish_state<V>(g.chain, t, E);
            if (live && g.dh0 && j == 0) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (in_range(b * g.D + d + v, g.batch * g.D)) g.dh0[b * g.D + d + v] = E[v];
            }
            continue;
        }

        const int64_t t0 = j * ROWS + w * S;
        const int own = w * S * 32 * V + lv;
        T *go = sm.rows[buf][0] + own, *ar = sm.rows[buf][1] + own, *ir = sm.rows[buf][2] + own, *u = sm.rows[buf][3] + own;
        float nab[V], nib[V], h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            nab[v] = live && g.a_bias && in_range(d + v, g.D) ? -kLog2e * __ldg(g.a_bias + d + v) : 0.f;
            nib[v] = live && g.i_bias && in_range(d + v, g.D) ? -kLog2e * __ldg(g.i_bias + d + v) : 0.f;
            const int64_t at = (b * g.chain.tiles + j) * g.D + d + v;
            h[v] = live && in_range(at, g.batch * g.chain.tiles * g.D) ? __ldg(g.ckpt_in + at) : 0.f;
        }
        if (kTma) {
            if (!mbar_wait(smem_u32(&sm.full[buf]), (it >> 1) & 1) && lane == 0) give_up(sm.c, 2u);
        } else {
            const int64_t r0 = j * ROWS, d0 = (int64_t)t.blk * 32 * V;
            fetch_rows<T, V, ROWS>(sm.rows[buf][0], g.dout, g, b, r0, d0);
            fetch_rows<T, V, ROWS>(sm.rows[buf][1], g.a_raw, g, b, r0, d0);
            fetch_rows<T, V, ROWS>(sm.rows[buf][2], g.i_raw, g, b, r0, d0);
            fetch_rows<T, V, ROWS>(sm.rows[buf][3], g.u, g, b, r0, d0);
            sync_work();
        }
        const float2 c = make_float2(sm.c.rate[buf][lv], sm.c.rate[buf][lv + V - 1]);
        const float2 na = make_float2(nab[0], nab[V - 1]), ni = make_float2(nib[0], nib[V - 1]);
        float a[S][V], x[S][V], r[S][V], i[S][V];
        auto out = [&](int k, float2 pa, float2 px, float2 pr, float2 pi) {
            set_pair<V, S>(a, k, pa);
            set_pair<V, S>(x, k, px);
            set_pair<V, S>(r, k, pr);
            set_pair<V, S>(i, k, pi);
        };
        const bool any = __any_sync(0xffffffffu, !(c.x < 0.25f && c.y < 0.25f));
        if (any) gate_terms<T, V, S, true>(c, na, ni, ar, ir, u, out);
        else gate_terms<T, V, S, false>(c, na, ni, ar, ir, u, out);
        // past the end dout is zero and so is every adjoint: those steps' terms are zeros by themselves
        float A[V], H[V], E[V];
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f, E[v] = 0.f;
#pragma unroll
        for (int k = 0; k < S; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                H[v] = fmaf(a[k][v], H[v], x[k][v]);
                A[v] *= a[k][v];
            }
#pragma unroll
        for (int k = S - 1; k >= 0; --k) {
            float gv[V];
            load_shared<V>(go + k * 32 * V, gv);
#pragma unroll
            for (int v = 0; v < V; ++v) E[v] = a[k][v] * (gv[v] + E[v]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sm.AH[w][lv + v] = make_float2(A[v], H[v]);
            sm.AE[w][lv + v] = make_float2(A[v], E[v]);
        }
        sync_maps();
        // while the adjoint is on its way: x[k] becomes the state h_{t-1}
        for (int q = 0; q < w; ++q) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 m = sm.AH[q][lv + v];
                h[v] = fmaf(m.x, h[v], m.y);
            }
        }
#pragma unroll
        for (int k = 0; k < S; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float hn = fmaf(a[k][v], h[v], x[k][v]);
                x[k][v] = h[v];
                h[v] = hn;
            }
        sync_state();
        // V = 1 computes its one element twice in the packed instructions
        float2 e, sl = splat(0.f), sa = splat(0.f), si = splat(0.f);
        {
            const float2 m0 = sm.AE[w][lv], m1 = sm.AE[w][lv + V - 1];
            e = make_float2(fmaf(m0.x, sm.c.in[lv], m0.y), fmaf(m1.x, sm.c.in[lv + V - 1], m1.y));
        }
#pragma unroll
        for (int k = S - 1; k >= 0; --k) {
            hold_loads();
            float uv[V], gv[V];
            load_shared<V>(u + k * 32 * V, uv);
            load_shared<V>(go + k * 32 * V, gv);
            const float2 pa = make_float2(a[k][0], a[k][V - 1]), pr = make_float2(r[k][0], r[k][V - 1]),
                         pi = make_float2(i[k][0], i[k][V - 1]), ph = make_float2(x[k][0], x[k][V - 1]),
                         pu = make_float2(uv[0], uv[V - 1]), pg = make_float2(gv[0], gv[V - 1]);
            const float2 s = mul2(c, pr);
            float2 am, om;
            if (any) decay2<true>(s, am, om);
            else decay2<false>(s, am, om);
            const float2 mi = rsqrt2(om);
            const float2 gt = add2(pg, e), iu = mul2(pi, pu), gm = mul2(gt, mul2(om, mi)), du = mul2(gm, pi);
            e = mul2(pa, gt);
            const float2 di = mul2(mul2(gm, iu), fma2(pi, splat(-1.f), splat(1.f)));
            // ds = e ((a / m) i u - h)
            const float2 ds = mul2(e, fma2(mul2(pa, mi), iu, mul2(ph, splat(-1.f))));
            const float2 da = mul2(mul2(ds, s), fma2(pr, splat(-1.f), splat(1.f)));
            sl = fma2(ds, pr, sl);
            sa = add2(sa, da);
            si = add2(si, di);
            const float ov[3][2] = {{da.x, da.y}, {di.x, di.y}, {du.x, du.y}};
            T* const to[3] = {ar, ir, u};
            T* const global[3] = {static_cast<T*>(g.da_raw), static_cast<T*>(g.di_raw), static_cast<T*>(g.du)};
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = ov[n][v];
                if (kTma) store_vec<V>(to[n] + k * 32 * V, o);
                else if (live && t0 + k < g.L) store_vec<V>(global[n] + (b * g.L + t0 + k) * g.D + d, o);
            }
        }
        if (kTma) fence_proxy_async();
        const float slv[2] = {sl.x, sl.y}, sav[2] = {sa.x, sa.y}, siv[2] = {si.x, si.y};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sm.red[0][w][lv + v] = slv[v];
            sm.red[1][w][lv + v] = sav[v];
            sm.red[2][w][lv + v] = siv[v];
        }
    }
    if (kTma && w == kWarps + 1 && lane == 0) {
        tma_store_wait_all();
        // every copy has been waited for, or is now: shared memory is given up with nothing in flight on it
        if (*reinterpret_cast<volatile int*>(&sm.c.gave_up))
            for (int k = 0; k < 2; ++k) mbar_drain(smem_u32(&sm.full[k]));
    }
}

// One token: V channels per thread, the rate worked out on the way.  64 x 5120 bf16: 3.5 us for 5 MB as a
// graph's node, a launch's own latency.
template <typename T, int V>
__global__ void __launch_bounds__(128) gated_step_kernel(GatedArgs g) {
    const int64_t cols = g.D / V;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t b = i / cols;
    if (b >= g.batch) return;
    const int64_t d = (i - b * cols) * V, at = b * g.D + d;
    float u[V], ar[V], ir[V], h[V];
    Vec<float, V> hs;
    hs.zero();
    const bool held = in_range(at, g.batch * g.D, V), params = in_range(d, g.D, V);
    if (held) hs.load_rw(g.state + at);
    load_vec<V>(static_cast<const T*>(g.u) + at, u);
    load_vec<V>(static_cast<const T*>(g.a_raw) + at, ar);
    load_vec<V>(static_cast<const T*>(g.i_raw) + at, ir);
    hs.get(h);
#pragma unroll
    for (int v = 0; v < V; v += 2) {
        // V = 1 computes its one element twice
        const int v1 = V == 1 ? 0 : v + 1;
        float2 r, i, a, om, nab = splat(0.f), nib = splat(0.f);
        if (g.a_bias && params) nab = make_float2(-kLog2e * __ldg(g.a_bias + d + v), -kLog2e * __ldg(g.a_bias + d + v1));
        if (g.i_bias && params) nib = make_float2(-kLog2e * __ldg(g.i_bias + d + v), -kLog2e * __ldg(g.i_bias + d + v1));
        const float2 c = !params ? splat(0.f)
                                 : make_float2(decay_rate(__ldg(g.Lam + d + v), g.rate), decay_rate(__ldg(g.Lam + d + v1), g.rate));
        gates2(make_float2(ar[v], ar[v1]), make_float2(ir[v], ir[v1]), nab, nib, r, i);
        decay2<true>(mul2(c, r), a, om);
        const float2 m = mul2(om, rsqrt2(om));
        const float2 hn = fma2(a, make_float2(h[v], h[v1]), mul2(mul2(m, i), make_float2(u[v], u[v1])));
        h[v] = hn.x;
        if (V > 1) h[v1] = hn.y;
    }
    hs.set(h);
    if (held) hs.store(g.state + at);
    store_vec<V>(static_cast<T*>(g.out) + at, h);
}

// Partial rows are [3][D]: dLam before its factor, da_bias, di_bias.
struct GatedGradPut {
    float *dLam, *da_bias, *di_bias;
    const float* Lam;
    float rate;
    int64_t D;
    __device__ void operator()(int64_t c, float s) const {
        const int64_t k = c / D, d = c - k * D;
        if (!in_range(d, D)) return;
        if (k == 0) dLam[d] = s * rate / (1.f + expf(-Lam[d]));
        else if (k == 1 && da_bias) da_bias[d] = s;
        else if (k == 2 && di_bias) di_bias[d] = s;
    }
};

// carry_in made to run out of polls, for a tile that waits for a map, a group and a state which nothing sets.
constexpr int kProbeTile = kFan * kFan + kFan + 1;
__device__ unsigned long long g_probe_words[32 * (kProbeTile + 1)];

__global__ void __launch_bounds__(32) carry_probe_kernel(unsigned int polls) {
    __shared__ ChainSmem s;
    for (int i = threadIdx.x; i < 32 * (kProbeTile + 1); i += 32) g_probe_words[i] = kUnset;
    __threadfence();
    __syncwarp();
    Chain c{};
    c.maps = c.groups = c.states = g_probe_words;
    c.tiles = c.ngroups = c.nsupers = kProbeTile + 1;
    c.cols = 1;
    const float first[1] = {0.f};
    float state[1];
    carry_in<1>(c, TileId{kProbeTile, 0, 0, 0}, first, state, s, 4u, polls);
}

// ---------------------------------------------------------------- host

sscan_status check_gated(const sscan_gated_problem* p) {
    if (!p) return api_fail(SSCAN_ERR_INVALID_ARG, "problem is NULL");
    if (p->batch < 0 || p->seqlen < 0 || p->dim < 0)
        return api_fail(SSCAN_ERR_INVALID_ARG, "negative size (batch %lld, seqlen %lld, dim %lld)",
                        (long long)p->batch, (long long)p->seqlen, (long long)p->dim);
    if (p->io_dtype != SSCAN_F32 && p->io_dtype != SSCAN_BF16)
        return api_fail(SSCAN_ERR_INVALID_ARG, "unknown io_dtype %d", (int)p->io_dtype);
    if (!(p->rate > 0.f) || p->rate > 1e6f)
        return api_fail(SSCAN_ERR_INVALID_ARG, "rate must be in (0, 1e6]");
    if (sscan_status s = api_elements(p->batch, p->seqlen, p->dim)) return s;
    // tickets are 32-bit counts of tiles (of 32 channels at least)
    // (and the steps of a sequence, which TMA coordinates count)
    const int64_t tiles = (p->seqlen + kCkpt - 1) / kCkpt, blocks = p->batch * ((p->dim + 31) / 32);
    if (tiles > 0 && blocks > ((int64_t(1) << 31) - 4096) / tiles)
        return api_fail(SSCAN_ERR_UNSUPPORTED, "more than 2^31 tiles of %d steps by 32 channels", kCkpt);
    if (p->seqlen > (int64_t(1) << 31) - 4096 || p->dim > (int64_t(1) << 31) - 4096 || p->batch > (int64_t(1) << 31) - 1)
        return api_fail(SSCAN_ERR_UNSUPPORTED, "a size of 2^31 or more");
    return SSCAN_OK;
}

int64_t gated_tiles(const sscan_gated_problem* p, int steps) {
    return (p->seqlen + kWarps * steps - 1) / (kWarps * steps);
}
int64_t gated_ckpts(const sscan_gated_problem* p) { return gated_tiles(p, kStepsBwd); }

// The chain's arrays, for column blocks of 32 channels or of 64, half as many of twice the width.
struct ChainLayout {
    size_t maps, groups, states, bytes;  // byte offsets, and the whole
};

ChainLayout chain_layout(const sscan_gated_problem* p, int steps) {
    ChainLayout l{};
    const size_t tiles = (size_t)gated_tiles(p, steps), words = (size_t)(p->batch * ((p->dim + 63) / 64 * 64)) * 8;
    if (tiles <= 1) return l;
    const size_t groups = (tiles + kFan - 1) / kFan, supers = (groups + kFan - 1) / kFan;
    l.maps = 256;  // the ticket before it
    l.groups = l.maps + words * tiles;
    l.states = l.groups + words * groups;
    l.bytes = round256(l.states + words * supers);
    return l;
}

size_t gated_ckpt_bytes(const sscan_gated_problem* p) {
    return round256((size_t)(p->batch * gated_ckpts(p) * p->dim) * sizeof(float));
}

bool empty(const sscan_gated_problem* p) { return p->batch == 0 || p->seqlen == 0 || p->dim == 0; }

cudaError_t set_chain(GatedArgs& g, const sscan_gated_problem* p, void* ws, int V, int steps, cudaStream_t st) {
    Chain& c = g.chain;
    c.tiles = gated_tiles(p, steps);
    g.nblk = (p->dim + 32 * V - 1) / (32 * V);
    c.cols = p->batch * g.nblk;
    c.ngroups = (c.tiles + kFan - 1) / kFan;
    c.nsupers = (c.ngroups + kFan - 1) / kFan;
    if (c.tiles <= 1) return cudaSuccess;
    const ChainLayout l = chain_layout(p, steps);
    char* base = static_cast<char*>(ws);
    c.ticket = reinterpret_cast<unsigned int*>(base);
    c.maps = reinterpret_cast<unsigned long long*>(base + l.maps);
    c.groups = reinterpret_cast<unsigned long long*>(base + l.groups);
    c.states = reinterpret_cast<unsigned long long*>(base + l.states);
    return cudaMemsetAsync(base, 0xff, l.bytes, st);
}

// A map over a (batch, L, D) tensor with boxes of `rows` steps by 32 V channels.
template <typename T, int V>
bool gated_map(CUtensorMap* m, const void* base, const GatedArgs& g, int rows) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)g.D, (cuuint64_t)g.L, (cuuint64_t)g.batch};
    const cuuint64_t strides[2] = {(cuuint64_t)(g.D * sizeof(T)), (cuuint64_t)(g.L * g.D * sizeof(T))};
    const cuuint32_t box[3] = {32 * V, (cuuint32_t)rows, 1}, each[3] = {1, 1, 1};
    return fn(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
              const_cast<void*>(base), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int V, bool kTma>
cudaError_t launch_gated(const GatedArgs& g, bool bwd, cudaStream_t st) {
    // as many blocks as the GPU holds at once; fewer tiles take fewer
    const int64_t all = g.chain.cols * g.chain.tiles, hold = (sizeof(T) == 2 ? 2 : 1) * kSmCount;
    const unsigned blocks = (unsigned)(all < hold ? all : hold);
    CUtensorMap m[7] = {};
    cudaError_t e;
    if (bwd) {
        const void* t[7] = {g.a_raw, g.i_raw, g.u, g.dout, g.da_raw, g.di_raw, g.du};
        if (kTma)
            for (int i = 0; i < 7; ++i)
                if (!gated_map<T, V>(&m[i], t[i], g, kWarps * kStepsBwd)) return cudaErrorInvalidValue;
        constexpr size_t smem = sizeof(GatedBwdSmem<T, V>);
        e = cudaFuncSetAttribute(gated_bwd_kernel<T, V, kTma>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        gated_bwd_kernel<T, V, kTma><<<blocks, kThreads, smem, st>>>(m[0], m[1], m[2], m[3], m[4], m[5], m[6], g);
    } else {
        const void* t[4] = {g.a_raw, g.i_raw, g.u, g.out ? g.out : g.u};
        if (kTma)
            for (int i = 0; i < 4; ++i)
                if (!gated_map<T, V>(&m[i], t[i], g, kWarps * kStepsFwd)) return cudaErrorInvalidValue;
        constexpr size_t smem = sizeof(GatedSmem<T, V, 3, kStepsFwd>);
        e = cudaFuncSetAttribute(gated_fwd_kernel<T, V, kTma>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        gated_fwd_kernel<T, V, kTma><<<blocks, kThreads, smem, st>>>(m[0], m[1], m[2], m[3], g);
    }
    api_count_launch();
    return cudaGetLastError();
}

// Two channels per lane where every pointer and the width allow it, by TMA where they are on
// 16-byte boundaries.
template <typename T>
cudaError_t launch_width(const GatedArgs& g, int V, bool tma, bool bwd, cudaStream_t st) {
    if (V == 1) return launch_gated<T, 1, false>(g, bwd, st);
    return tma ? launch_gated<T, 2, true>(g, bwd, st) : launch_gated<T, 2, false>(g, bwd, st);
}

sscan_status run_gated(GatedArgs& g, const sscan_gated_problem* p, void* ws, bool bwd, cudaStream_t st) {
    const size_t es = p->io_dtype == SSCAN_BF16 ? 2 : 4;
    auto all_aligned = [&](size_t n) {
        for (const void* q : {g.u, g.a_raw, g.i_raw, (const void*)g.out, g.dout, (const void*)g.du,
                              (const void*)g.da_raw, (const void*)g.di_raw})
            if (!aligned_to(q, n)) return false;
        return g.D * es % n == 0;
    };
    const int V = all_aligned(2 * es) ? 2 : 1;
    cudaError_t e = set_chain(g, p, ws, V, bwd ? kStepsBwd : kStepsFwd, st);
    if (e != cudaSuccess) return api_fail(SSCAN_ERR_CUDA, "clearing the carry's words: %s", cudaGetErrorString(e));
    const bool tma = all_aligned(16);
    e = es == 2 ? launch_width<__nv_bfloat16>(g, V, tma, bwd, st) : launch_width<float>(g, V, tma, bwd, st);
    if (e != cudaSuccess)
        return api_fail(SSCAN_ERR_CUDA, "gated %s kernel: %s", bwd ? "backward" : "forward", cudaGetErrorString(e));
    return SSCAN_OK;
}

GatedArgs gated_args(const sscan_gated_problem* p, const void* u, const void* a_raw, const void* i_raw,
                     const float* Lam, const float* a_bias, const float* i_bias, const float* h0) {
    GatedArgs g{};
    g.batch = p->batch, g.L = p->seqlen, g.D = p->dim, g.rate = p->rate;
    g.u = u, g.a_raw = a_raw, g.i_raw = i_raw;
    g.Lam = Lam, g.a_bias = a_bias, g.i_bias = i_bias, g.h0 = h0;
    return g;
}

template <typename T, int V>
void step_blocks(const GatedArgs& g, cudaStream_t st) {
    const int64_t n = g.batch * (g.D / V);
    gated_step_kernel<T, V><<<(unsigned)((n + 127) / 128), 128, 0, st>>>(g);
}

}  // namespace

cudaError_t launch_carry_probe(unsigned int polls, cudaStream_t st) {
    carry_probe_kernel<<<1, 32, 0, st>>>(polls);
    return cudaGetLastError();
}

cudaError_t read_device_error_gated(unsigned int* value, int clear) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error_gated, sizeof(unsigned int));
    if (e == cudaSuccess && clear && *value) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_device_error_gated, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace sscan

using namespace sscan;

extern "C" {

int64_t sscan_gated_checkpoints(const sscan_gated_problem* p) {
    return check_gated(p) == SSCAN_OK ? gated_ckpts(p) : 0;
}

size_t sscan_gated_workspace_size(const sscan_gated_problem* p, int op) {
    if (check_gated(p) != SSCAN_OK || empty(p)) return 0;
    const size_t fwd = chain_layout(p, kStepsFwd).bytes, bwd = chain_layout(p, kStepsBwd).bytes;
    if (op == SSCAN_OP_FWD) return fwd;
    if (op != SSCAN_OP_BWD) return 0;
    // the carry, one row of partial sums per tile, and the checkpoints when the caller has none
    return (fwd > bwd ? fwd : bwd) + round256((size_t)(p->batch * gated_ckpts(p) * 3 * p->dim) * sizeof(float)) +
           gated_ckpt_bytes(p);
}

sscan_status sscan_gated_fwd(const sscan_gated_problem* p, const void* u, const void* a_raw, const void* i_raw,
                             const float* Lam, const float* a_bias, const float* i_bias, const float* h0, void* out,
                             float* h_last, float* checkpoints, void* workspace, size_t workspace_bytes,
                             void* stream) {
    api_begin();
    if (sscan_status s = check_gated(p)) return s;
    if (p->batch == 0 || p->dim == 0) return SSCAN_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->seqlen == 0) {
        if (!h_last) return SSCAN_OK;
        const size_t bytes = (size_t)(p->batch * p->dim) * sizeof(float);
        const cudaError_t e = h0 ? cudaMemcpyAsync(h_last, h0, bytes, cudaMemcpyDeviceToDevice, st)
                                 : cudaMemsetAsync(h_last, 0, bytes, st);
        return e == cudaSuccess ? SSCAN_OK : api_fail(SSCAN_ERR_CUDA, "copying h0 to h_last: %s", cudaGetErrorString(e));
    }
    if (!u || !a_raw || !i_raw || !Lam || !out)
        return api_fail(SSCAN_ERR_INVALID_ARG, "u, a_raw, i_raw, Lam and out are required");
    if (sscan_status s = api_workspace(sscan_gated_workspace_size(p, SSCAN_OP_FWD), workspace, workspace_bytes)) return s;
    GatedArgs g = gated_args(p, u, a_raw, i_raw, Lam, a_bias, i_bias, h0);
    g.out = out, g.h_last = h_last, g.ckpt = checkpoints;
    return run_gated(g, p, workspace, false, st);
}

sscan_status sscan_gated_bwd(const sscan_gated_problem* p, const void* u, const void* a_raw, const void* i_raw,
                             const float* Lam, const float* a_bias, const float* i_bias, const float* h0,
                             const float* checkpoints, const void* dout, void* du, void* da_raw, void* di_raw,
                             float* dLam, float* da_bias, float* di_bias, float* dh0, void* workspace,
                             size_t workspace_bytes, void* stream) {
    api_begin();
    if (sscan_status s = check_gated(p)) return s;
    if (p->dim == 0) return SSCAN_OK;
    if (!dLam) return api_fail(SSCAN_ERR_INVALID_ARG, "dLam is required");
    if (da_bias && !a_bias) return api_fail(SSCAN_ERR_INVALID_ARG, "da_bias needs a_bias");
    if (di_bias && !i_bias) return api_fail(SSCAN_ERR_INVALID_ARG, "di_bias needs i_bias");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (empty(p)) {  // sums over nothing
        cudaError_t e = cudaSuccess;
        for (float* q : {dLam, da_bias, di_bias})
            if (e == cudaSuccess && q) e = cudaMemsetAsync(q, 0, (size_t)p->dim * sizeof(float), st);
        if (e == cudaSuccess && dh0 && p->batch)
            e = cudaMemsetAsync(dh0, 0, (size_t)(p->batch * p->dim) * sizeof(float), st);
        return e == cudaSuccess ? SSCAN_OK : api_fail(SSCAN_ERR_CUDA, "zeroing gradients: %s", cudaGetErrorString(e));
    }
    if (!u || !a_raw || !i_raw || !Lam || !dout || !du || !da_raw || !di_raw)
        return api_fail(SSCAN_ERR_INVALID_ARG, "u, a_raw, i_raw, Lam, dout, du, da_raw and di_raw are required");
    if (sscan_status s = api_workspace(sscan_gated_workspace_size(p, SSCAN_OP_BWD), workspace, workspace_bytes)) return s;
    const size_t fwd = chain_layout(p, kStepsFwd).bytes, bwd = chain_layout(p, kStepsBwd).bytes;
    const size_t chain = fwd > bwd ? fwd : bwd;
    float* ckpt = reinterpret_cast<float*>(static_cast<char*>(workspace) + chain);
    GatedArgs g = gated_args(p, u, a_raw, i_raw, Lam, a_bias, i_bias, h0);
    if (!checkpoints) {
        g.ckpt = ckpt;
        if (sscan_status s = run_gated(g, p, workspace, false, st)) return s;
        g.ckpt = nullptr;
    }
    g.ckpt_in = checkpoints ? checkpoints : ckpt;
    g.part = reinterpret_cast<float*>(reinterpret_cast<char*>(ckpt) + gated_ckpt_bytes(p));
    g.dout = dout, g.du = du, g.da_raw = da_raw, g.di_raw = di_raw, g.dh0 = dh0;
    if (sscan_status s = run_gated(g, p, workspace, true, st)) return s;
    launch_rowsum(g.part, p->batch * gated_ckpts(p), 3 * p->dim,
                  GatedGradPut{dLam, da_bias, di_bias, Lam, p->rate, p->dim}, st);
    api_count_launch();
    return api_launched("gated gradient sum");
}

sscan_status sscan_gated_step(const sscan_gated_problem* p, const void* u, const void* a_raw, const void* i_raw,
                              const float* Lam, const float* a_bias, const float* i_bias, float* state, void* out,
                              void* stream) {
    api_begin();
    if (sscan_status s = check_gated(p)) return s;
    if (p->seqlen != 1)
        return api_fail(SSCAN_ERR_INVALID_ARG, "sscan_gated_step takes seqlen == 1, got %lld", (long long)p->seqlen);
    if (p->batch == 0 || p->dim == 0) return SSCAN_OK;
    if (!u || !a_raw || !i_raw || !Lam || !state || !out)
        return api_fail(SSCAN_ERR_INVALID_ARG, "u, a_raw, i_raw, Lam, state and out are required");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    GatedArgs g = gated_args(p, u, a_raw, i_raw, Lam, a_bias, i_bias, nullptr);
    g.out = out, g.state = state;
    const bool bf16 = p->io_dtype == SSCAN_BF16;
    const size_t es = bf16 ? 2 : 4;
    const bool four = p->dim % 4 == 0 && aligned_to(u, 4 * es) && aligned_to(a_raw, 4 * es) &&
                      aligned_to(i_raw, 4 * es) && aligned_to(out, 4 * es) && aligned_to(state, 16);
    if (bf16) four ? step_blocks<__nv_bfloat16, 4>(g, st) : step_blocks<__nv_bfloat16, 1>(g, st);
    else four ? step_blocks<float, 4>(g, st) : step_blocks<float, 1>(g, st);
    api_count_launch();
    return api_launched("gated step kernel");
}

}  // extern "C"
