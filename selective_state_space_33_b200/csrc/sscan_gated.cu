// sscan_gated.cu -- the gated linear recurrence with one state per channel,
//   r = sigmoid(a_raw + a_bias),  i = sigmoid(i_raw + i_bias),  s = rate softplus(Lam) r,
//   a = exp(-s),  m = sqrt(1 - a^2),   h_t = a_t h_{t-1} + m_t i_t u_t,   out_t = h_t,
// for every (batch, channel); its backward pass and its one-token step.
//
// One pass over the sequence.  A block owns a tile of kTile steps by 32 V channels: each of
// its kWarps warps scans kSteps consecutive steps from zero with the gates' results in
// registers, the warps' affine maps h -> A h + H are combined through shared memory, the
// state entering the tile comes from the tiles before it, and a second sweep over the
// registers writes the outputs.  So every input is read once and every output written once,
// however the sequence is split.
//
// The carry between tiles (chain_carry): tiles take their place in line from an atomic
// ticket in time order, so all tiles a block waits for have already started.  A tile
// publishes its own map as soon as it has it; the state entering a group of kGroup tiles is
// handed on by the last tile of the group before.  A tile composes the maps of its group's
// earlier tiles, in order, and applies them to the group's state: the grouping is fixed, so
// two runs round alike, and the serial chain has one hop per kGroup * kTile steps.
#include <cuda_runtime.h>

#include <cstddef>

#include "sscan_check.cuh"
#include "sscan_host.h"
#include "sscan_launch.h"
#include "sscan_math.cuh"
#include "sscan_rowsum.cuh"
#include "sscan_vec.cuh"

namespace sscan {

__device__ unsigned int g_device_error_gated = 0;

namespace {

constexpr int kWarps = 8;
constexpr int kSteps = 8;                // steps per warp
constexpr int kTile = kWarps * kSteps;   // steps per block; also the checkpoint interval
constexpr int kGroup = 32;               // tiles per hop of the serial chain
constexpr uint32_t kPollLimit = 1u << 22;

struct Chain {
    unsigned int* ticket;   // null: one tile per sequence, no carry
    unsigned int* mapped;   // [cols][tiles] 1 once the tile's map is published
    unsigned int* entered;  // [cols][groups] 1 once the group's entering state is published
    float2* maps;           // [cols][tiles][32 V] (A, H)
    float* states;          // [cols][groups][32 V]
    int64_t tiles, groups, cols;
};

struct GatedArgs {
    int64_t batch, L, D, nblk;  // nblk: channel blocks of 32 V
    const void *u, *a_raw, *i_raw;
    const float *Lam, *a_bias, *i_bias, *h0;
    float rate;
    void* out;       // (batch, L, D) or null (checkpoints only)
    float* h_last;   // (batch, D) or null
    float* ckpt;     // (batch, tiles, D) or null: the state entering each tile
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

// expm1(-s) for 0 <= s < 1/4: Taylor series to s^6, the dropped s^7/5040 below 1.3e-8 relative.
__device__ __forceinline__ float expm1_neg(float s) {
    const float p = fmaf(s, fmaf(s, fmaf(s, fmaf(s, fmaf(s, 1.f / 720.f, -1.f / 120.f), 1.f / 24.f), -1.f / 6.f), 0.5f), -1.f);
    return s * p;
}

// a = exp(-s) and 1 - a^2 = -e (2 + e), e = expm1(-s).  Near s = 0 both come from the series:
// the difference 1 - a would cancel, and a long memory multiplies a's error by its length.
__device__ __forceinline__ void decay(float s, float& a, float& om) {
    const float ea = ex2(-s * kLog2e);
    const float e = s < 0.25f ? expm1_neg(s) : ea - 1.f;
    a = 1.f + e;
    om = -e * (2.f + e);
}

__device__ __forceinline__ float sqrt_fast(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rsqrt_fast(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// rate * softplus(Lam), once per channel of a block
__device__ __forceinline__ float decay_rate(float lam, float rate) {
    return rate * (lam > 20.f ? lam : log1pf(expf(lam)));
}

__device__ __forceinline__ unsigned int load_acquire(const unsigned int* p) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void store_release(unsigned int* p, unsigned int v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

__device__ __forceinline__ bool wait_set(const unsigned int* p) {
    for (uint32_t i = 0; i < kPollLimit; ++i) {
        if (load_acquire(p)) return true;
        __nanosleep(32);
    }
    return false;
}

// One warp: the state entering tile k (in chain order) of column block `col`, for the V
// channels of each lane, from the tile's own map (A, H) and the state `first` entering tile 0.
// A wait that gives up raises `err` and goes on, publishing as if it had not, so that no
// later tile waits for it in turn.
template <int V>
__device__ __forceinline__ void chain_carry(const Chain& c, int64_t col, int64_t k, const float (&A)[V],
                                            const float (&H)[V], const float (&first)[V], float (&state)[V],
                                            unsigned int err) {
    const int lane = threadIdx.x & 31;
    const int64_t g = k / kGroup, k0 = g * kGroup;
    const int n = (int)(k - k0);
    const bool more = k + 1 < c.tiles, closes = n == kGroup - 1;
    const int64_t nmaps = c.cols * c.tiles * 32 * V, nstates = c.cols * c.groups * 32 * V;
    if (more && !closes) {
        const int64_t at = ((col * c.tiles + k) * 32 + lane) * V;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (in_range(at + v, nmaps)) __stcg(c.maps + at + v, make_float2(A[v], H[v]));
        __threadfence();
        __syncwarp();
        if (lane == 0) store_release(c.mapped + col * c.tiles + k, 1u);
    }
    float Ac[V], Hc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) Ac[v] = 1.f, Hc[v] = 0.f, state[v] = first[v];
    bool ok = true;
    if (n > 0) {
        if (lane < n) ok = wait_set(c.mapped + col * c.tiles + k0 + lane);
        __syncwarp();
        __threadfence();
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const int64_t at = ((col * c.tiles + k0 + i) * 32 + lane) * V;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 m = in_range(at + v, nmaps) ? __ldcg(c.maps + at + v) : make_float2(0.f, 0.f);
                Ac[v] *= m.x;
                Hc[v] = fmaf(m.x, Hc[v], m.y);
            }
        }
    }
    if (g > 0) {
        if (lane == 0) ok = wait_set(c.entered + col * c.groups + g) && ok;
        __syncwarp();
        __threadfence();
        const int64_t at = ((col * c.groups + g) * 32 + lane) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) state[v] = in_range(at + v, nstates) ? __ldcg(c.states + at + v) : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) state[v] = fmaf(Ac[v], state[v], Hc[v]);
    if (more && closes) {
        const int64_t at = ((col * c.groups + g + 1) * 32 + lane) * V;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (in_range(at + v, nstates)) __stcg(c.states + at + v, fmaf(A[v], state[v], H[v]));
        __threadfence();
        __syncwarp();
        if (lane == 0) store_release(c.entered + col * c.groups + g + 1, 1u);
    }
    if (!ok) atomicOr(&g_device_error_gated, err);
}

// This block's place in line: tickets run through the column blocks first, then the tiles.
__device__ __forceinline__ void take_ticket(const Chain& c, int64_t& col, int64_t& k) {
    __shared__ unsigned int place;
    if (threadIdx.x == 0) place = c.ticket ? atomicAdd(c.ticket, 1u) : blockIdx.x;
    __syncthreads();
    k = place / c.cols;
    col = place - k * c.cols;
}

template <typename T, int V>
__global__ void __launch_bounds__(32 * kWarps) gated_fwd_kernel(GatedArgs g) {
    __shared__ float sA[kWarps][32 * V], sH[kWarps][32 * V], sIn[32 * V], sRate[32 * V];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t col, j;
    take_ticket(g.chain, col, j);
    const int64_t b = col / g.nblk, d = ((col - b * g.nblk) * 32 + lane) * V;
    const bool live = d < g.D;  // V divides D, so a lane's channels are all inside or all outside
    const int64_t t0 = j * kTile + w * kSteps;

    Vec<T, V> u[kSteps], ar[kSteps], ir[kSteps];
    const int64_t base = (b * g.L + t0) * g.D + d;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
        if (live && t0 + k < g.L) {
            ar[k].load(static_cast<const T*>(g.a_raw) + base + k * g.D);
            ir[k].load(static_cast<const T*>(g.i_raw) + base + k * g.D);
            u[k].load(static_cast<const T*>(g.u) + base + k * g.D);
        }
    if (w < V) {  // channel x of the block, x = 0 .. 32 V - 1
        const int64_t x = (col - b * g.nblk) * 32 * V + threadIdx.x;
        sRate[threadIdx.x] = x < g.D ? decay_rate(__ldg(g.Lam + x), g.rate) : 0.f;
    }
    float ab[V], ib[V], first[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        ab[v] = live && g.a_bias ? __ldg(g.a_bias + d + v) : 0.f;
        ib[v] = live && g.i_bias ? __ldg(g.i_bias + d + v) : 0.f;
        first[v] = live && g.h0 && w == 0 ? __ldg(g.h0 + b * g.D + d + v) : 0.f;
    }
    __syncthreads();
    float a[kSteps][V], x[kSteps][V], A[V], H[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        float uv[V], av[V], iv[V];
        u[k].get(uv);
        ar[k].get(av);
        ir[k].get(iv);
        const bool in = live && t0 + k < g.L;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float om;
            decay(sRate[lane * V + v] * sigmoid(av[v] + ab[v]), a[k][v], om);
            x[k][v] = sqrt_fast(om) * sigmoid(iv[v] + ib[v]) * uv[v];
            if (!in) a[k][v] = 1.f, x[k][v] = 0.f;  // past the end: the identity map
            H[v] = fmaf(a[k][v], H[v], x[k][v]);
            A[v] *= a[k][v];
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) sA[w][lane * V + v] = A[v], sH[w][lane * V + v] = H[v];
    __syncthreads();
    if (w == 0) {
        float state[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.f, H[v] = 0.f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) {
                H[v] = fmaf(sA[q][lane * V + v], H[v], sH[q][lane * V + v]);
                A[v] *= sA[q][lane * V + v];
            }
        }
        if (g.chain.ticket) {
            chain_carry<V>(g.chain, col, j, A, H, first, state, 1u);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) state[v] = first[v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) sIn[lane * V + v] = state[v];
        if (live) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (g.ckpt) g.ckpt[(b * g.chain.tiles + j) * g.D + d + v] = state[v];
                if (g.h_last && j == g.chain.tiles - 1) g.h_last[b * g.D + d + v] = fmaf(A[v], state[v], H[v]);
            }
        }
    }
    if (!g.out) return;
    __syncthreads();
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = sIn[lane * V + v];
        for (int q = 0; q < w; ++q) h[v] = fmaf(sA[q][lane * V + v], h[v], sH[q][lane * V + v]);
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(a[k][v], h[v], x[k][v]);
        if (live && t0 + k < g.L) store_vec<V>(static_cast<T*>(g.out) + base + k * g.D, h);
    }
}

// The adjoint e_t that step t hands to h_{t-1} is affine in the one it gets: with
// g_t = dout_t + e_{t+1},  e_t = a_t g_t.  Tiles run from the last to the first; the state
// entering a tile is known (a checkpoint), so the forward states are rebuilt without a wait.
//   du = g m i,   di_raw = g m i u (1 - i),
//   ds = -e_t (h_{t-1} - (a / m) i u),   da_raw = ds s (1 - r),   dLam = sum ds r * rate sigmoid(Lam)
// Where s underflows to 0, m = 0 and its slope's limit is not finite; that term is left out.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kWarps, 2) gated_bwd_kernel(GatedArgs g) {
    __shared__ float sA[kWarps][32 * V], sH[kWarps][32 * V], sE[kWarps][32 * V], sIn[32 * V], sRate[32 * V];
    __shared__ float red[3][kWarps][32 * V];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t col, rank;
    take_ticket(g.chain, col, rank);
    const int64_t j = g.chain.tiles - 1 - rank;
    const int64_t b = col / g.nblk, d = ((col - b * g.nblk) * 32 + lane) * V;
    const bool live = d < g.D;
    const int64_t t0 = j * kTile + w * kSteps;

    Vec<T, V> u[kSteps], ar[kSteps], ir[kSteps], go[kSteps];
    const int64_t base = (b * g.L + t0) * g.D + d;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
        if (live && t0 + k < g.L) {
            ar[k].load(static_cast<const T*>(g.a_raw) + base + k * g.D);
            go[k].load(static_cast<const T*>(g.dout) + base + k * g.D);
            ir[k].load(static_cast<const T*>(g.i_raw) + base + k * g.D);
            u[k].load(static_cast<const T*>(g.u) + base + k * g.D);
        }
    if (w < V) {
        const int64_t x = (col - b * g.nblk) * 32 * V + threadIdx.x;
        sRate[threadIdx.x] = x < g.D ? decay_rate(__ldg(g.Lam + x), g.rate) : 0.f;
    }
    float ab[V], ib[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        ab[v] = live && g.a_bias ? __ldg(g.a_bias + d + v) : 0.f;
        ib[v] = live && g.i_bias ? __ldg(g.i_bias + d + v) : 0.f;
        h[v] = live ? __ldg(g.ckpt_in + (b * g.chain.tiles + j) * g.D + d + v) : 0.f;
    }
    __syncthreads();
    float a[kSteps][V], x[kSteps][V], r[kSteps][V], i[kSteps][V], A[V], H[V], E[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f, E[v] = 0.f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        float uv[V], av[V], iv[V];
        u[k].get(uv);
        ar[k].get(av);
        ir[k].get(iv);
        const bool in = live && t0 + k < g.L;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float om;
            r[k][v] = sigmoid(av[v] + ab[v]);
            i[k][v] = sigmoid(iv[v] + ib[v]);
            decay(sRate[lane * V + v] * r[k][v], a[k][v], om);
            x[k][v] = sqrt_fast(om) * i[k][v] * uv[v];
            if (!in) a[k][v] = 1.f, x[k][v] = 0.f;
            H[v] = fmaf(a[k][v], H[v], x[k][v]);
            A[v] *= a[k][v];
        }
    }
#pragma unroll
    for (int k = kSteps - 1; k >= 0; --k) {
        float gv[V];
        go[k].get(gv);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (live && t0 + k < g.L) E[v] = a[k][v] * (gv[v] + E[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sA[w][lane * V + v] = A[v];
        sH[w][lane * V + v] = H[v];
        sE[w][lane * V + v] = E[v];
    }
    __syncthreads();
    if (w == 0) {
        float state[V], zero[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.f, E[v] = 0.f, zero[v] = 0.f;
#pragma unroll
            for (int q = kWarps - 1; q >= 0; --q) {
                E[v] = fmaf(sA[q][lane * V + v], E[v], sE[q][lane * V + v]);
                A[v] *= sA[q][lane * V + v];
            }
        }
        if (g.chain.ticket) {
            chain_carry<V>(g.chain, col, rank, A, E, zero, state, 2u);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) state[v] = 0.f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sIn[lane * V + v] = state[v];
            if (live && g.dh0 && j == 0) g.dh0[b * g.D + d + v] = fmaf(A[v], state[v], E[v]);
        }
    }
    // meanwhile the other warps rebuild the states: x[k] becomes h_{t-1}
#pragma unroll
    for (int v = 0; v < V; ++v)
        for (int q = 0; q < w; ++q) h[v] = fmaf(sA[q][lane * V + v], h[v], sH[q][lane * V + v]);
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float hn = fmaf(a[k][v], h[v], x[k][v]);
            x[k][v] = h[v];
            h[v] = hn;
        }
    __syncthreads();
    float e[V], sl[V], sa[V], si[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        e[v] = sIn[lane * V + v];
        for (int q = kWarps - 1; q > w; --q) e[v] = fmaf(sA[q][lane * V + v], e[v], sE[q][lane * V + v]);
        sl[v] = sa[v] = si[v] = 0.f;
    }
#pragma unroll
    for (int k = kSteps - 1; k >= 0; --k) {
        if (!live || t0 + k >= g.L) continue;
        float uv[V], gv[V], du[V], da[V], di[V];
        u[k].get(uv);
        go[k].get(gv);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float s = sRate[lane * V + v] * r[k][v];
            float am, om;
            decay(s, am, om);
            const float mi = om > 0.f ? rsqrt_fast(om) : 0.f;  // 1 / m
            const float gt = gv[v] + e[v];
            e[v] = a[k][v] * gt;
            du[v] = gt * (om * mi) * i[k][v];
            di[v] = du[v] * uv[v] * (1.f - i[k][v]);
            const float ds = -e[v] * (x[k][v] - am * mi * i[k][v] * uv[v]);
            da[v] = ds * s * (1.f - r[k][v]);
            sl[v] = fmaf(ds, r[k][v], sl[v]);
            sa[v] += da[v];
            si[v] += di[v];
        }
        store_vec<V>(static_cast<T*>(g.du) + base + k * g.D, du);
        store_vec<V>(static_cast<T*>(g.da_raw) + base + k * g.D, da);
        store_vec<V>(static_cast<T*>(g.di_raw) + base + k * g.D, di);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        red[0][w][lane * V + v] = sl[v];
        red[1][w][lane * V + v] = sa[v];
        red[2][w][lane * V + v] = si[v];
    }
    __syncthreads();
    if (w < 3 && live) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) s += red[w][q][lane * V + v];
            g.part[((b * g.chain.tiles + j) * 3 + w) * g.D + d + v] = s;
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(128) gated_step_kernel(GatedArgs g) {
    const int64_t cols = g.D / V;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t b = i / cols;
    if (b >= g.batch) return;
    const int64_t d = (i - b * cols) * V, at = b * g.D + d;
    float u[V], ar[V], ir[V], h[V];
    Vec<float, V> hs;
    hs.load_rw(g.state + at);
    load_vec<V>(static_cast<const T*>(g.u) + at, u);
    load_vec<V>(static_cast<const T*>(g.a_raw) + at, ar);
    load_vec<V>(static_cast<const T*>(g.i_raw) + at, ir);
    hs.get(h);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float a, om;
        const float ab = g.a_bias ? __ldg(g.a_bias + d + v) : 0.f, ib = g.i_bias ? __ldg(g.i_bias + d + v) : 0.f;
        decay(decay_rate(__ldg(g.Lam + d + v), g.rate) * sigmoid(ar[v] + ab), a, om);
        h[v] = fmaf(a, h[v], sqrt_fast(om) * sigmoid(ir[v] + ib) * u[v]);
    }
    hs.set(h);
    hs.store(g.state + at);
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
        if (k == 0) dLam[d] = s * rate / (1.f + expf(-Lam[d]));
        else if (k == 1 && da_bias) da_bias[d] = s;
        else if (k == 2 && di_bias) di_bias[d] = s;
    }
};

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
    const int64_t tiles = (p->seqlen + kTile - 1) / kTile, blocks = p->batch * ((p->dim + 31) / 32);
    if (tiles > 0 && blocks > ((int64_t(1) << 31) - 1) / tiles)
        return api_fail(SSCAN_ERR_UNSUPPORTED, "more than 2^31 tiles of %d steps by 32 channels", kTile);
    return SSCAN_OK;
}

int64_t gated_tiles(const sscan_gated_problem* p) { return (p->seqlen + kTile - 1) / kTile; }

// The chain's arrays for column blocks of 32 channels (the most there can be): counters first,
// since they are cleared together before each launch.  Channel blocks of 64 use the same
// space, half as many columns of twice the width.
struct ChainLayout {
    size_t counters, maps, states, bytes;  // byte offsets and total
};

ChainLayout chain_layout(const sscan_gated_problem* p) {
    ChainLayout l{};
    const size_t tiles = (size_t)gated_tiles(p), cols = (size_t)(p->batch * ((p->dim + 63) / 64 * 2));
    if (tiles <= 1) return l;
    const size_t groups = (tiles + kGroup - 1) / kGroup;
    l.counters = round256((1 + cols * (tiles + groups)) * sizeof(unsigned int));
    l.maps = l.counters;
    l.states = l.maps + round256(cols * tiles * 32 * sizeof(float2));
    l.bytes = l.states + round256(cols * groups * 32 * sizeof(float));
    return l;
}

size_t gated_ckpt_bytes(const sscan_gated_problem* p) {
    return round256((size_t)(p->batch * gated_tiles(p) * p->dim) * sizeof(float));
}

bool empty(const sscan_gated_problem* p) { return p->batch == 0 || p->seqlen == 0 || p->dim == 0; }

// Two channels per lane where every pointer and the width allow it.
int gated_width(const GatedArgs& g, size_t es) {
    if (g.D % 2) return 1;
    for (const void* p : {g.u, g.a_raw, g.i_raw, (const void*)g.out, g.dout, (const void*)g.du,
                          (const void*)g.da_raw, (const void*)g.di_raw})
        if (!aligned_to(p, 2 * es)) return 1;
    return 2;
}

cudaError_t set_chain(GatedArgs& g, const sscan_gated_problem* p, void* ws, int V, cudaStream_t st) {
    Chain& c = g.chain;
    c.tiles = gated_tiles(p);
    g.nblk = (p->dim + 32 * V - 1) / (32 * V);
    c.cols = p->batch * g.nblk;
    c.groups = (c.tiles + kGroup - 1) / kGroup;
    if (c.tiles <= 1) return cudaSuccess;
    const ChainLayout l = chain_layout(p);
    char* base = static_cast<char*>(ws);
    c.ticket = reinterpret_cast<unsigned int*>(base);
    c.mapped = c.ticket + 1;
    c.entered = c.mapped + c.cols * c.tiles;
    c.maps = reinterpret_cast<float2*>(base + l.maps);
    c.states = reinterpret_cast<float*>(base + l.states);
    return cudaMemsetAsync(base, 0, l.counters, st);
}

template <typename T>
void launch_gated(const GatedArgs& g, bool bwd, int V, cudaStream_t st) {
    const unsigned blocks = (unsigned)(g.chain.cols * g.chain.tiles);
    if (bwd) {
        if (V == 2) gated_bwd_kernel<T, 2><<<blocks, 32 * kWarps, 0, st>>>(g);
        else gated_bwd_kernel<T, 1><<<blocks, 32 * kWarps, 0, st>>>(g);
    } else {
        if (V == 2) gated_fwd_kernel<T, 2><<<blocks, 32 * kWarps, 0, st>>>(g);
        else gated_fwd_kernel<T, 1><<<blocks, 32 * kWarps, 0, st>>>(g);
    }
    api_count_launch();
}

sscan_status run_gated(GatedArgs& g, const sscan_gated_problem* p, void* ws, bool bwd, cudaStream_t st) {
    const bool bf16 = p->io_dtype == SSCAN_BF16;
    const int V = gated_width(g, bf16 ? 2 : 4);
    const cudaError_t e = set_chain(g, p, ws, V, st);
    if (e != cudaSuccess) return api_fail(SSCAN_ERR_CUDA, "clearing the carry's counters: %s", cudaGetErrorString(e));
    if (bf16) launch_gated<__nv_bfloat16>(g, bwd, V, st);
    else launch_gated<float>(g, bwd, V, st);
    return api_launched(bwd ? "gated backward kernel" : "gated forward kernel");
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
    return check_gated(p) == SSCAN_OK ? gated_tiles(p) : 0;
}

size_t sscan_gated_workspace_size(const sscan_gated_problem* p, int op) {
    if (check_gated(p) != SSCAN_OK || empty(p)) return 0;
    const size_t chain = chain_layout(p).bytes;
    if (op == SSCAN_OP_FWD) return chain;
    if (op != SSCAN_OP_BWD) return 0;
    // the carry, one row of partial sums per tile, and the checkpoints when the caller has none
    return chain + round256((size_t)(p->batch * gated_tiles(p) * 3 * p->dim) * sizeof(float)) + gated_ckpt_bytes(p);
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
    const size_t chain = chain_layout(p).bytes;
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
    launch_rowsum(g.part, p->batch * gated_tiles(p), 3 * p->dim,
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
