// sscan_conv.cu -- the causal depthwise convolution of the block's input branch,
//   y_t = bias + sum_k W[k] x_{t-K+1+k},   out_t = SiLU(y_t) or y_t,   K = 2 .. 4,
// for every (batch, channel), with the K-1 inputs before the sequence as its state;
// its backward pass and its one-token step.
//
// Every element is read and written once, against K multiply-adds and (with SiLU) two
// special-function operations, so all three are bound by HBM bandwidth.  A thread owns V
// neighbouring channels (4 or 2 elements in one access where width and pointers allow it) and
// walks a stretch of steps with the window in registers; the loads of several rows are issued
// before any of them is used.
#include <cuda_runtime.h>

#include <initializer_list>

#include "sscan_check.cuh"
#include "sscan_host.h"
#include "sscan_math.cuh"
#include "sscan_plan.h"
#include "sscan_rowsum.cuh"
#include "sscan_vec.cuh"

namespace sscan {
namespace {

struct ConvArgs {
    int64_t batch, L, D;
    const void* u;        // (batch, L, D)
    const float* w;       // (D, K)
    const float* bias;    // (D) or null
    const void* state0;   // (batch, K-1, D) or null
    void* out;            // (batch, L, D)
    void* last;           // (batch, K-1, D) or null
    int64_t tile;         // steps per thread, a multiple of kAhead
    int wide_w;           // weight on a 16-byte boundary
    // backward
    const void* dout;     // (batch, L, D)
    void* du;             // (batch, L, D)
    void* dstate0;        // (batch, K-1, D) or null
    float* part;          // [batch * tiles][K + 1][D] partial sums of dW and dbias
    int64_t tiles;
};

constexpr int kAhead = 8;

// The window's row at time t < L: from the sequence, the state, or zero before both.
template <typename T, int K, int V>
__device__ __forceinline__ void load_row(const ConvArgs& a, int64_t b, int64_t t, int64_t d, float (&x)[V]) {
    if (t >= 0) {
        load_vec<V>(static_cast<const T*>(a.u) + (b * a.L + t) * a.D + d, x);
    } else if (a.state0 && in_range((b * (K - 1) + t + K - 1) * a.D + d, a.batch * (K - 1) * a.D, V)) {
        load_vec<V>(static_cast<const T*>(a.state0) + (b * (K - 1) + t + K - 1) * a.D + d, x);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = 0.f;
    }
}

// Rows of the weight come in one access each where they are aligned to their size.
template <int K, int V>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int64_t d, float (&w)[K][V], float (&bias)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float* p = a.w + (d + v) * K;
        const bool in = in_range((d + v) * K, a.D * K, K);
        if (!in) {
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][v] = 0.f;
        } else if (K == 4 && a.wide_w) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(p));
            w[0][v] = f.x, w[1][v] = f.y, w[K - 2][v] = f.z, w[K - 1][v] = f.w;
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][v] = __ldg(p + k);
        }
        bias[v] = a.bias && in_range(d + v, a.D) ? __ldg(a.bias + d + v) : 0.f;
    }
}

// One thread: V channels of one batch row, `tile` steps.  Threads run along the channels
// first, so that a warp's accesses are consecutive.  8 x 2048 x 1536 bf16, 4 taps, SiLU: 25 us,
// 4.0 TB/s; what is left over the 15.4 us of its bytes is the latency of one wave of threads.
template <typename T, int K, int V, bool kSilu>
__global__ void __launch_bounds__(128, 8) conv_fwd_kernel(ConvArgs a) {
    const int64_t cols = a.D / V;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t row = i / cols;
    if (row >= a.batch * a.tiles) return;
    const int64_t d = (i - row * cols) * V, b = row / a.tiles, t0 = (row - b * a.tiles) * a.tile;
    const int64_t left = a.L - t0;
    int n = (int)(left < a.tile ? left : a.tile);

    float w[K][V], bias[V], x[K - 1][V];
    load_taps<K, V>(a, d, w, bias);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) load_row<T, K, V>(a, b, t0 - (K - 1) + k, d, x[k]);
    const T* up = static_cast<const T*>(a.u) + (b * a.L + t0) * a.D + d;
    T* op = static_cast<T*>(a.out) + (b * a.L + t0) * a.D + d;
    auto step = [&](const Vec<T, V>& in) {
        float xn[V], y[V];
        in.get(xn);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float s = fmaf(w[K - 1][v], xn[v], bias[v]);
#pragma unroll
            for (int k = 0; k < K - 1; ++k) s = fmaf(w[k][v], x[k][v], s);
            y[v] = kSilu ? silu(s) : s;
#pragma unroll
            for (int k = 0; k < K - 2; ++k) x[k][v] = x[k + 1][v];
            x[K - 2][v] = xn[v];
        }
        store_vec<V>(op, y);
        op += a.D;
    };
    constexpr int N = V * sizeof(T) > 8 ? kAhead / 2 : kAhead;  // at most 64 bytes of loads ahead
#pragma unroll 1
    for (; n >= N; n -= N) {
        Vec<T, V> in[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            in[j].load(up);
            up += a.D;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) step(in[j]);
    }
    if (n > 0) {
        Vec<T, V> in[N];
#pragma unroll
        for (int j = 0; j < N - 1; ++j)
            if (j < n) in[j].load(up + j * a.D);
#pragma unroll
        for (int j = 0; j < N - 1; ++j)
            if (j < n) step(in[j]);
    }
    if (a.last && t0 + a.tile >= a.L) {
        // the window now holds the last K - 1 inputs; each was read exactly, so this is a copy
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
            if (in_range((b * (K - 1) + k) * a.D + d, a.batch * (K - 1) * a.D, V))
                store_vec<V>(static_cast<T*>(a.last) + (b * (K - 1) + k) * a.D + d, x[k]);
    }
}

constexpr int kBwdGroups = 8;  // stretches per block, whose dW partials the block adds up

// dy_t = dout_t act'(y_t);  dx_t = sum_k W[k] dy_{t+K-1-k};  dW[k] = sum_t dy_t x_{t-K+1+k}.
// A block is 32 lanes of V channels by kBwdGroups stretches of `tile` steps; each thread runs
// K-1 steps past its stretch to have every dy its dx needs (recomputed, not exchanged: two
// rows in `tile`), and the block writes one row of dW and dbias partial sums.  3 x 1021 x 1531 fp32
// (an odd width: one channel per thread): 21 us, 2.7 TB/s.
template <typename T, int K, int V, bool kSilu>
__global__ void __launch_bounds__(32 * kBwdGroups, 3) conv_bwd_kernel(ConvArgs a) {
    __shared__ float red[kBwdGroups][(K + 1) * V][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int64_t d = ((int64_t)blockIdx.x * 32 + lane) * V;
    const int64_t b = blockIdx.y / a.tiles, slot = blockIdx.y - b * a.tiles;
    const int64_t t0 = (slot * kBwdGroups + grp) * a.tile;
    float sums[K + 1][V];
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) sums[k][v] = 0.f;
    if (d < a.D && t0 < a.L) {
        const int64_t t1 = t0 + a.tile < a.L ? t0 + a.tile : a.L;  // the stretch whose dx this thread writes
        float w[K][V], bias[V], x[K][V], dy[K][V];
        load_taps<K, V>(a, d, w, bias);
#pragma unroll
        for (int k = 0; k < K - 1; ++k) load_row<T, K, V>(a, b, t0 - (K - 1) + k, d, x[k + 1]);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) dy[k][v] = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) x[0][v] = 0.f;
        const T* up = static_cast<const T*>(a.u) + (b * a.L + t0) * a.D + d;
        const T* gp = static_cast<const T*>(a.dout) + (b * a.L + t0) * a.D + d;
        T* dp = static_cast<T*>(a.du) + (b * a.L + t0) * a.D + d;
        const int own = (int)(t1 - t0);                      // steps of this stretch
        const int have = (int)(a.L - t0 < own + K - 1 ? a.L - t0 : own + K - 1);  // and those there are past it
        // step s of the stretch: dy_s, its share of dW, and dx of K - 1 steps earlier
        auto step = [&](int s, const Vec<T, V>& in, const Vec<T, V>& gin) {
            float xn[V], gv[V], dx[V];
            in.get(xn);
            gin.get(gv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int k = 0; k < K - 1; ++k) {
                    x[k][v] = x[k + 1][v];
                    dy[k][v] = dy[k + 1][v];
                }
                x[K - 1][v] = xn[v];
                float dyt = gv[v];
                if (kSilu) {
                    float y = bias[v];
#pragma unroll
                    for (int k = 0; k < K; ++k) y = fmaf(w[k][v], x[k][v], y);
                    dyt *= dsilu(y);
                }
                if (s >= have) dyt = 0.f;                    // past the sequence
                dy[K - 1][v] = dyt;
                if (s < own) {
#pragma unroll
                    for (int k = 0; k < K; ++k) sums[k][v] = fmaf(dyt, x[k][v], sums[k][v]);
                    sums[K][v] += dyt;
                }
                // dy[j] is dy_{s-K+1+j}; dx_{s-K+1} = sum_k W[k] dy_{s-k}
                dx[v] = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) dx[v] = fmaf(w[k][v], dy[K - 1 - k][v], dx[v]);
            }
            if (s >= K - 1) {
                store_vec<V>(dp, dx);
                dp += a.D;
            } else if (t0 == 0 && a.dstate0 && in_range((b * (K - 1) + s) * a.D + d, a.batch * (K - 1) * a.D, V)) {
                store_vec<V>(static_cast<T*>(a.dstate0) + (b * (K - 1) + s) * a.D + d, dx);
            }
        };
        constexpr int N = 4;
        int s = 0;
#pragma unroll 1
        for (; s + N <= have; s += N) {
            Vec<T, V> in[N], gin[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                in[j].load(up);
                gin[j].load(gp);
                up += a.D;
                gp += a.D;
            }
#pragma unroll
            for (int j = 0; j < N; ++j) step(s + j, in[j], gin[j]);
        }
#pragma unroll 1
        for (; s < own + K - 1; ++s) {
            Vec<T, V> in, gin;
            in.zero();
            gin.zero();
            if (s < have) {
                in.load(up);
                gin.load(gp);
                up += a.D;
                gp += a.D;
            }
            step(s, in, gin);
        }
    }
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) red[grp][k * V + v][lane] = sums[k][v];
    __syncthreads();
    for (int k = grp; k <= K; k += kBwdGroups) {
        float s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = 0.f;
#pragma unroll
            for (int g = 0; g < kBwdGroups; ++g) s[v] += red[g][k * V + v][lane];
        }
        if (d < a.D) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t at = ((int64_t)blockIdx.y * (K + 1) + k) * a.D + d + v;
                if (in_range(at, a.batch * a.tiles * (K + 1) * a.D)) a.part[at] = s[v];
            }
        }
    }
}

// One token: the window is the state; shift it in place.  64 x 5120 bf16, 4 taps: 2.8-3.5 us for 5 MB
// as a graph's node, a launch's own latency; two channels per thread (four 3.5-4.2 us, one 3.5).
template <typename T, int K, int V, bool kSilu>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvArgs a) {
    const int64_t cols = a.D / V;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t b = i / cols;
    if (b >= a.batch) return;
    const int64_t d = (i - b * cols) * V;
    T* sp = static_cast<T*>(a.last) + b * (K - 1) * a.D + d;
    auto held = [&](int k) { return in_range((b * (K - 1) + k) * a.D + d, a.batch * (K - 1) * a.D, V); };
    Vec<T, V> in[K];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        in[k].zero();
        if (held(k)) in[k].load_rw(sp + k * a.D);
    }
    in[K - 1].load(static_cast<const T*>(a.u) + b * a.D + d);
    float w[K][V], y[V];
    load_taps<K, V>(a, d, w, y);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float x[V];
        in[k].get(x);
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = fmaf(w[k][v], x[v], y[v]);
    }
    if (kSilu) {
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = silu(y[v]);
    }
    store_vec<V>(static_cast<T*>(a.out) + b * a.D + d, y);
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
        if (held(k)) in[k + 1].store(sp + k * a.D);
}

// Partial rows are [K + 1][D]: K columns of dweight (D, K), then dbias (D).
struct ConvGradPut {
    float* dweight;
    float* dbias;  // or null
    int64_t D, K;
    __device__ void operator()(int64_t c, float s) const {
        const int64_t k = c / D, d = c - k * D;
        if (k < K) {
            if (in_range(d * K + k, D * K)) dweight[d * K + k] = s;
        } else if (dbias && in_range(d, D)) {
            dbias[d] = s;
        }
    }
};

// ---------------------------------------------------------------- host

enum { kConvFwd, kConvBwd, kConvStep };

template <typename T, int K, int V, bool kSilu>
void launch_one(int op, const ConvArgs& a, cudaStream_t st) {
    if constexpr (V <= 2) if (op == kConvBwd) {
        const dim3 grid((unsigned)((a.D / V + 31) / 32), (unsigned)(a.batch * a.tiles));
        conv_bwd_kernel<T, K, V, kSilu><<<grid, 32 * kBwdGroups, 0, st>>>(a);
        return;
    }
    const int64_t n = (op == kConvFwd ? a.batch * a.tiles : a.batch) * (a.D / V);
    const unsigned blocks = (unsigned)((n + 127) / 128);
    if (op == kConvFwd) conv_fwd_kernel<T, K, V, kSilu><<<blocks, 128, 0, st>>>(a);
    else if constexpr (V <= 2) conv_step_kernel<T, K, V, kSilu><<<blocks, 128, 0, st>>>(a);
}

template <typename T, int K, int V>
void launch_silu(int op, const ConvArgs& a, bool act, cudaStream_t st) {
    if (act) launch_one<T, K, V, true>(op, a, st);
    else launch_one<T, K, V, false>(op, a, st);
}

template <typename T, int V>
void launch_taps(int op, const ConvArgs& a, int taps, bool act, cudaStream_t st) {
    if (taps == 2) launch_silu<T, 2, V>(op, a, act, st);
    else if (taps == 3) launch_silu<T, 3, V>(op, a, act, st);
    else launch_silu<T, 4, V>(op, a, act, st);
}

// The widest access that the width and every pointer allow, up to 4 channels in the forward
// pass and 2 elsewhere: the backward keeps 3 K + 2 fp32 values per channel in registers, and a
// step has so few elements that it wants more threads rather than wider ones.
int conv_width(int op, int64_t D, size_t es, std::initializer_list<const void*> ptrs) {
    for (int v = op == kConvFwd ? 4 : 2; v > 1; v /= 2) {
        bool ok = D % v == 0;
        for (const void* p : ptrs) ok = ok && aligned_to(p, v * es);
        if (ok) return v;
    }
    return 1;
}

template <typename T>
void launch_width(int op, const ConvArgs& a, int v, int taps, bool act, cudaStream_t st) {
    if (v == 4) launch_taps<T, 4>(op, a, taps, act, st);
    else if (v == 2) launch_taps<T, 2>(op, a, taps, act, st);
    else launch_taps<T, 1>(op, a, taps, act, st);
}

void launch_conv(int op, ConvArgs a, int taps, bool act, bool bf16, cudaStream_t st) {
    a.wide_w = aligned_to(a.w, 16);
    const int v = conv_width(op, a.D, bf16 ? 2 : 4, {a.u, a.state0, a.out, a.last, a.dout, a.du, a.dstate0});
    if (bf16) launch_width<__nv_bfloat16>(op, a, v, taps, act, st);
    else launch_width<float>(op, a, v, taps, act, st);
    api_count_launch();
}

sscan_status check_conv(const sscan_conv_problem* p) {
    if (!p) return api_fail(SSCAN_ERR_INVALID_ARG, "problem is NULL");
    if (p->batch < 0 || p->seqlen < 0 || p->dim < 0)
        return api_fail(SSCAN_ERR_INVALID_ARG, "negative size (batch %lld, seqlen %lld, dim %lld)",
                        (long long)p->batch, (long long)p->seqlen, (long long)p->dim);
    if (p->taps < 1) return api_fail(SSCAN_ERR_INVALID_ARG, "taps must be >= 1");
    if (p->taps < 2 || p->taps > 4)
        return api_fail(SSCAN_ERR_UNSUPPORTED, "taps %lld outside 2..4", (long long)p->taps);
    if (p->io_dtype != SSCAN_F32 && p->io_dtype != SSCAN_BF16)
        return api_fail(SSCAN_ERR_INVALID_ARG, "unknown io_dtype %d", (int)p->io_dtype);
    if (p->flags & ~SSCAN_CONV_SILU)
        return api_fail(SSCAN_ERR_INVALID_ARG, "unknown flag bits 0x%x", (unsigned)(p->flags & ~SSCAN_CONV_SILU));
    // thread and block counts of the kernels below stay within 31 bits
    return api_elements(p->batch, p->seqlen, p->dim);
}

// Steps per thread, a multiple of kAhead from 8 to 48: what makes one wave of threads (8 blocks of
// 128 per SM), so that small problems spread out and large ones re-read few rows (K-1 per
// stretch).  8 x 2048 x 1536 bf16: 25.2 us at the 48 this gives, 26.5, 28.0 and 27.4 at 24, 32, 64.
int64_t conv_fwd_tile(const sscan_conv_problem* p) {
    const int64_t n = (p->batch * p->seqlen * ((p->dim + 3) / 4) / (kSmCount * 1024) + kAhead - 1) / kAhead * kAhead;
    return n < kAhead ? kAhead : n > 48 ? 48 : n;
}

// The backward's stretch: 32 steps; blocks (of kBwdGroups stretches) along one sequence are
// kept to 65535 / batch by longer stretches, whatever the length.
int64_t conv_bwd_tile(const sscan_conv_problem* p, int64_t* tiles) {
    int64_t tile = 32;
    while (p->batch * ((p->seqlen + tile * kBwdGroups - 1) / (tile * kBwdGroups)) > 65535 && tile < p->seqlen) tile *= 2;
    *tiles = (p->seqlen + tile * kBwdGroups - 1) / (tile * kBwdGroups);
    return tile;
}

size_t conv_part_floats(const sscan_conv_problem* p) {
    int64_t tiles;
    conv_bwd_tile(p, &tiles);
    return (size_t)(p->batch * tiles * (p->taps + 1) * p->dim);
}

}  // namespace
}  // namespace sscan

using namespace sscan;

extern "C" {

size_t sscan_conv_workspace_size(const sscan_conv_problem* p, int op) {
    if (check_conv(p) != SSCAN_OK || op != SSCAN_OP_BWD) return 0;
    if (p->batch == 0 || p->seqlen == 0 || p->dim == 0 || p->batch > 65535) return 0;
    return round256(conv_part_floats(p) * sizeof(float));
}

sscan_status sscan_conv_fwd(const sscan_conv_problem* p, const void* u, const float* weight, const float* bias,
                            const void* state0, void* out, void* state_last, void* stream) {
    api_begin();
    if (sscan_status s = check_conv(p)) return s;
    if (p->batch == 0 || p->dim == 0) return SSCAN_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->seqlen == 0) {
        if (!state_last) return SSCAN_OK;
        const size_t bytes = (size_t)(p->batch * (p->taps - 1) * p->dim) * (p->io_dtype == SSCAN_BF16 ? 2 : 4);
        const cudaError_t e = state0 ? cudaMemcpyAsync(state_last, state0, bytes, cudaMemcpyDeviceToDevice, st)
                                     : cudaMemsetAsync(state_last, 0, bytes, st);
        return e == cudaSuccess ? SSCAN_OK
                                : api_fail(SSCAN_ERR_CUDA, "copying state0 to state_last: %s", cudaGetErrorString(e));
    }
    if (!u || !weight || !out) return api_fail(SSCAN_ERR_INVALID_ARG, "u, weight and out are required");
    ConvArgs a{};
    a.batch = p->batch, a.L = p->seqlen, a.D = p->dim;
    a.u = u, a.w = weight, a.bias = bias, a.state0 = state0, a.out = out, a.last = state_last;
    a.tile = conv_fwd_tile(p);
    a.tiles = (a.L + a.tile - 1) / a.tile;
    launch_conv(kConvFwd, a, (int)p->taps, p->flags & SSCAN_CONV_SILU, p->io_dtype == SSCAN_BF16, st);
    return api_launched("convolution kernel");
}

sscan_status sscan_conv_bwd(const sscan_conv_problem* p, const void* u, const float* weight, const float* bias,
                            const void* state0, const void* dout, void* du, float* dweight, float* dbias,
                            void* dstate0, void* workspace, size_t workspace_bytes, void* stream) {
    api_begin();
    if (sscan_status s = check_conv(p)) return s;
    if (p->dim == 0) return SSCAN_OK;
    if (!dweight) return api_fail(SSCAN_ERR_INVALID_ARG, "dweight is required");
    if (dbias && !bias) return api_fail(SSCAN_ERR_INVALID_ARG, "dbias needs bias");
    if (dstate0 && !state0) return api_fail(SSCAN_ERR_INVALID_ARG, "dstate0 needs state0");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->batch == 0 || p->seqlen == 0) {  // sums over nothing
        cudaError_t e = cudaMemsetAsync(dweight, 0, (size_t)(p->dim * p->taps) * sizeof(float), st);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)p->dim * sizeof(float), st);
        const size_t bytes = (size_t)(p->batch * (p->taps - 1) * p->dim) * (p->io_dtype == SSCAN_BF16 ? 2 : 4);
        if (e == cudaSuccess && dstate0 && bytes) e = cudaMemsetAsync(dstate0, 0, bytes, st);
        return e == cudaSuccess ? SSCAN_OK : api_fail(SSCAN_ERR_CUDA, "zeroing gradients: %s", cudaGetErrorString(e));
    }
    if (p->batch > 65535) return api_fail(SSCAN_ERR_UNSUPPORTED, "batch %lld > 65535", (long long)p->batch);
    if (!u || !weight || !dout || !du)
        return api_fail(SSCAN_ERR_INVALID_ARG, "u, weight, dout and du are required");
    if (sscan_status s = api_workspace(sscan_conv_workspace_size(p, SSCAN_OP_BWD), workspace, workspace_bytes)) return s;
    ConvArgs a{};
    a.batch = p->batch, a.L = p->seqlen, a.D = p->dim;
    a.u = u, a.w = weight, a.bias = bias, a.state0 = state0;
    a.dout = dout, a.du = du, a.dstate0 = dstate0, a.part = static_cast<float*>(workspace);
    a.tile = conv_bwd_tile(p, &a.tiles);
    launch_conv(kConvBwd, a, (int)p->taps, p->flags & SSCAN_CONV_SILU, p->io_dtype == SSCAN_BF16, st);
    if (sscan_status s = api_launched("convolution backward kernel")) return s;
    launch_rowsum(a.part, a.batch * a.tiles, (p->taps + 1) * a.D, ConvGradPut{dweight, dbias, a.D, p->taps}, st);
    api_count_launch();
    return api_launched("convolution gradient sum");
}

sscan_status sscan_conv_step(const sscan_conv_problem* p, const void* u, const float* weight, const float* bias,
                             void* state, void* out, void* stream) {
    api_begin();
    if (sscan_status s = check_conv(p)) return s;
    if (p->seqlen != 1)
        return api_fail(SSCAN_ERR_INVALID_ARG, "sscan_conv_step takes seqlen == 1, got %lld", (long long)p->seqlen);
    if (p->batch == 0 || p->dim == 0) return SSCAN_OK;
    if (!u || !weight || !state || !out)
        return api_fail(SSCAN_ERR_INVALID_ARG, "u, weight, state and out are required");
    ConvArgs a{};
    a.batch = p->batch, a.L = 1, a.D = p->dim;
    a.u = u, a.w = weight, a.bias = bias, a.out = out, a.last = state;
    launch_conv(kConvStep, a, (int)p->taps, p->flags & SSCAN_CONV_SILU, p->io_dtype == SSCAN_BF16,
                static_cast<cudaStream_t>(stream));
    return api_launched("convolution step kernel");
}

}  // extern "C"
