// sscan_heads.cuh -- what the forward and backward kernels of the multi-head recurrence share.
//
// Per batch row and head, with dl = softplus(delta_raw + bias), q = dl A, w = expm1(q) / A:
//   S_t = exp(q_t) S_{t-1} + w_t u_t B_t^T   (P x N),    y_t = S_t C_t + D u_t,
//   out_t = y_t SiLU(z_t).
// A chunk of kQ steps, with c_t the running sum of q from the chunk's start and S the state
// entering it, is three matrix products:
//   Y = M U + exp(c) C S^T,   M_ts = (C_t . B_s) exp(c_t - c_s) w_s for s <= t, else 0,
//   S' = exp(c_end) S + (f U)^T B,   f_s = exp(c_end - c_s) w_s.
#pragma once

#include <cuda_runtime.h>

#include "sscan_check.cuh"
#include "sscan_host.h"
#include "sscan_launch.h"
#include "sscan_math.cuh"
#include "sscan_mma.cuh"
#include "sscan_tma.cuh"

namespace sscan {

constexpr int kQ = 64;        // steps per chunk
constexpr int kHeadDim = 64;  // a head's channels in a tile (fewer are padded with zeros)

struct HeadsArgs {
    int64_t batch, L;
    int H, P, N, G;
    int softplus;
    int vec;                  // rows of u, z, dout and of B, C start and end on 16-byte boundaries
    const void *u, *delta_raw, *B, *C, *z;
    const float *A, *bias, *D, *h0;
    void* out;
    float* h_last;
    int64_t chunks;           // ceil(L / kQ)
    // sequence split into segments of seg_chunks chunks
    int64_t seg_chunks, nseg;
    float* states;            // [batch][H][nseg][P][N]: segment end states, then entering states
    float* decays;            // [batch][H][nseg]: sum of q over the segment
    // segments handed on instead (the output pass alone): states is then the state after each, and
    unsigned int* ticket;     // null, or the place in line of the next block
    unsigned int* handed;     // [batch][H][nseg] 1 once that state is there
};

// Extents of the arrays below, in elements, and head h's entry of a parameter (0 without one).
__device__ __forceinline__ int64_t state_extent(const HeadsArgs& a) { return a.batch * a.H * a.P * a.N; }
__device__ __forceinline__ int64_t states_extent(const HeadsArgs& a) { return a.nseg * state_extent(a); }
__device__ __forceinline__ int64_t segments(const HeadsArgs& a) { return a.batch * a.H * a.nseg; }
__device__ __forceinline__ float head_param(const HeadsArgs& a, const float* p, int h) {
    return p && in_range(h, a.H) ? __ldg(p + h) : 0.f;
}

// Scalars of one chunk's steps, and their running sums (read two at a time, hence the alignment).
template <int Q>
struct alignas(16) ChunkScalarsOf {
    float ch[Q], cl[Q];     // log2(e) c_t as the sum of two floats: the difference of two of
                              // them keeps its absolute error near 2^-24 whatever c_t's size
    float w[Q];
    float e[Q];               // exp(c_t)
    float d[Q];               // exp(c_end - c_t)
    float f[Q];               // d_t w_t
    float total;              // c_end
};
using ChunkScalars = ChunkScalarsOf<kQ>;

// What the gradients of the scalars need besides.
struct ChunkSteps {
    float dl[kQ], raw[kQ];    // step sizes, and what softplus was taken of
};

// One warp fills s (and steps) for steps t0 .. t0 + Q - 1 of (b, h); past L: q = w = 0.
template <typename T, int Q>
__device__ __forceinline__ void chunk_scalars(ChunkScalarsOf<Q>& s, const HeadsArgs& a, int64_t b, int h, int64_t t0,
                                              ChunkSteps* steps = nullptr) {
    constexpr int PER = Q / 32;  // consecutive steps of a lane
    const int lane = threadIdx.x & 31;
    const float A = head_param(a, a.A, h), bias = head_param(a, a.bias, h);
    const T* dr = static_cast<const T*>(a.delta_raw);
    double c[PER];
    float w[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t t = t0 + PER * lane + i;
        c[i] = 0.0;
        w[i] = 0.f;
        if (steps) steps->dl[PER * lane + i] = steps->raw[PER * lane + i] = 0.f;
        if (t < a.L) {
            const float r = IO<T>::load(dr, (b * a.L + t) * a.H + h) + bias;
            const float dl = a.softplus ? (r > 20.f ? r : log1pf(expf(r))) : r;
            const float q = dl * A;
            w[i] = A != 0.f ? expm1f(q) / A : dl;
            c[i] = q < -1e4f ? -1e4 : (double)q;  // exp(-1e4) is 0 in fp32; keeps sums finite
            if (steps) steps->dl[PER * lane + i] = dl, steps->raw[PER * lane + i] = r;
        }
        if (i) c[i] += c[i - 1];
    }
    double run = c[PER - 1];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const double v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += v;
    }
    // (not run - c[PER - 1]: a NaN in a lane's later step would reach its earlier ones)
    double before = __shfl_up_sync(0xffffffffu, run, 1);
    if (lane == 0) before = 0.0;
    const double end = __shfl_sync(0xffffffffu, run, 31);
    constexpr double l2e = 1.4426950408889634074;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int t = PER * lane + i;
        const double ct = (before + c[i]) * l2e;
        s.ch[t] = (float)ct;
        s.cl[t] = (float)(ct - (double)s.ch[t]);
        s.w[t] = w[i];
        s.e[t] = ex2((float)ct);
        s.d[t] = ex2((float)(end * l2e - ct));
        s.f[t] = s.d[t] * w[i];
    }
    if (lane == 0) s.total = (float)end;
}

// exp(c_t - c_s)
template <int Q>
__device__ __forceinline__ float chunk_decay(const ChunkScalarsOf<Q>& s, int t, int u) {
    return ex2((s.ch[t] - s.ch[u]) + (s.cl[t] - s.cl[u]));
}

// rows x COLS tile of T from global rows (`stride` elements apart) into shared memory, zeros
// past `rows` and `cols`.  vec: every row starts on a 16-byte boundary and cols is a multiple
// of 16 bytes.
template <typename T, int COLS>
__device__ __forceinline__ void load_tile(T* dst, int pitch, const T* src, int64_t stride, int64_t rows, int cols,
                                          bool vec, int tid, int threads) {
    constexpr int VE = 16 / sizeof(T), PER = COLS / VE;
    for (int i = tid; i < kQ * PER; i += threads) {
        const int r = i / PER, c = (i - r * PER) * VE;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < rows && c < cols) {
            const T* p = src + r * stride + c;
            if (vec) {
                v = __ldg(reinterpret_cast<const uint4*>(p));
            } else {
                T* e = reinterpret_cast<T*>(&v);
#pragma unroll
                for (int j = 0; j < VE; ++j)
                    if (c + j < cols) e[j] = p[j];
            }
        }
        *reinterpret_cast<uint4*>(dst + r * pitch + c) = v;
    }
}

// The same by cp.async where vec allows it; the caller commits and waits.
template <typename T, int COLS>
__device__ __forceinline__ void load_tile_async(T* dst, int pitch, const T* src, int64_t stride, int64_t rows, int cols,
                                                bool vec, int tid, int threads) {
    if (!vec) {
        load_tile<T, COLS>(dst, pitch, src, stride, rows, cols, false, tid, threads);
        return;
    }
    constexpr int VE = 16 / sizeof(T), PER = COLS / VE;
    for (int i = tid; i < kQ * PER; i += threads) {
        const int r = i / PER, c = (i - r * PER) * VE;
        const bool in = r < rows && c < cols;
        cp_async16(dst + r * pitch + c, in ? src + r * stride + c : src, in);
    }
}

// 16 rows of kHeadDim elements by one warp, likewise.
template <typename T>
__device__ __forceinline__ void load_rows_async(T* dst, int pitch, const T* src, int64_t stride, int64_t rows, int cols,
                                                bool vec) {
    constexpr int VE = 16 / sizeof(T), PER = kHeadDim / VE;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = lane; i < 16 * PER; i += 32) {
        const int r = i / PER, c = (i - r * PER) * VE;
        if (vec) {
            const bool in = r < rows && c < cols;
            cp_async16(dst + r * pitch + c, in ? src + r * stride + c : src, in);
        } else {
#pragma unroll
            for (int j = 0; j < VE; ++j) dst[r * pitch + c + j] = r < rows && c + j < cols ? src[r * stride + c + j] : from_f32<T>(0.f);
        }
    }
}

// Neighbouring values x, y in the tile type: fp32 as they are; bf16 as two parts, which keep 16
// bits (a relative 2^-17), and what they leave, rounded to a third (24 bits).
template <typename T>
__device__ __forceinline__ uint32_t split_store2(T* hi, T* lo, int at, float x, float y) {
    if constexpr (Mma<T>::kExact32) {
        *reinterpret_cast<float2*>(hi + at) = make_float2(x, y);
        return 0u;
    } else {
        const uint32_t h = Mma<T>::pack(x, y);
        *reinterpret_cast<uint32_t*>(hi + at) = h;
        x -= __uint_as_float(h << 16);
        y -= __uint_as_float(h & 0xffff0000u);
        const uint32_t l = Mma<T>::pack(x, y);
        *reinterpret_cast<uint32_t*>(lo + at) = l;
        return Mma<T>::pack(x - __uint_as_float(l << 16), y - __uint_as_float(l & 0xffff0000u));
    }
}

template <typename T, int NT> struct HeadsPitch {
    static constexpr int P = kHeadDim + Mma<T>::PAD;
    static constexpr int N = NT + Mma<T>::PAD;
    static constexpr int Q = kQ + Mma<T>::PAD;
};

// A thread's elements (p, n) = place(j), j < COUNT <= 64, of the state after steps t0 .. t1 - 1 of (b, h), as it
// has just stored them to `dest`: those that are not finite are taken again from the state `first` before t0
// (null: zero), step by step.  A chunk's products split their operands in parts, and an infinity in one of
// them is not a number there, where the recurrence has an infinity.  An infinity is not decayed here, since
// exp(q) may underflow.
template <typename T, int COUNT, typename Place>
static __device__ __noinline__ void state_by_steps(float* dest, Place place, const HeadsArgs& a, int64_t b, int h, int64_t t0,
                                                   int64_t t1, const float* first) {
    const int grp = h / (a.H / a.G);
    const int64_t extent = (int64_t)a.P * a.N;
    const float A = head_param(a, a.A, h), bias = head_param(a, a.bias, h);
    float S[COUNT];
    unsigned long long redo = 0;
#pragma unroll 1
    for (int j = 0; j < COUNT; ++j) {
        const int2 at = place(j);
        const int64_t i = (int64_t)at.x * a.N + at.y;
        if (at.x >= a.P || at.y >= a.N || !in_range(i, extent) || fabsf(__ldcg(dest + i)) <= 3.4e38f) continue;
        redo |= 1ull << j;
        S[j] = first ? __ldcg(first + i) : 0.f;
    }
    unsigned long long todo = redo;
#pragma unroll 1
    for (int64_t t = t0; t < t1 && todo; ++t) {
        const int64_t tok = b * a.L + t;
        const float r = IO<T>::load(static_cast<const T*>(a.delta_raw), tok * a.H + h) + bias;
        const float dl = a.softplus ? (r > 20.f ? r : log1pf(expf(r))) : r;
        const float q = dl * A, e = ex2(q * kLog2e), w = A != 0.f ? expm1f(q) / A : dl;
#pragma unroll 1
        for (unsigned long long left = todo; left; left &= left - 1) {
            const int j = __ffsll((long long)left) - 1;
            const int2 at = place(j);
            const float x = w * IO<T>::load(static_cast<const T*>(a.u), (tok * a.H + h) * a.P + at.x) *
                            IO<T>::load(static_cast<const T*>(a.B), (tok * a.G + grp) * a.N + at.y);
            S[j] = fmaf(fabsf(S[j]) > 3.4e38f ? 1.f : e, S[j], x);
            if (S[j] != S[j]) todo &= ~(1ull << j);  // and it stays so
        }
    }
#pragma unroll 1
    for (; redo; redo &= redo - 1) {
        const int j = __ffsll((long long)redo) - 1;
        const int2 at = place(j);
        __stcg(dest + (int64_t)at.x * a.N + at.y, S[j]);
    }
}

// Whether any of a thread's elements is not finite.
template <int COUNT>
__device__ __forceinline__ bool not_finite(const float (&v)[COUNT]) {
    float probe = 0.f;
#pragma unroll
    for (int j = 0; j < COUNT; ++j) probe = fmaf(v[j], 0.f, probe);
    return probe != 0.f;
}

// Segment end states from zero (forward: of S; reverse: of its adjoint), and the carry
// through them; sscan_heads.cu.
void launch_heads_carry(const HeadsArgs& a, bool reverse, const float* first, float* last, cudaStream_t st);
sscan_status check_heads(const sscan_heads_problem* p);
HeadsArgs heads_args(const sscan_heads_problem* p, const void* u, const void* delta_raw, const float* delta_bias,
                     const float* A, const void* B, const void* C, const float* D_skip, const void* z,
                     const float* h0);
// The forward on tcgen05 (sscan_heads_tc.cu): bf16, more than 32 states, rows on 16-byte boundaries.
// Its chunks are 128 steps; a.chunks, seg_chunks and nseg count those.
constexpr int kTcQ = 128;
cudaError_t launch_heads_tc(const HeadsArgs& a, bool local, cudaStream_t st);


// Local states of every segment: forward (u, B) or, with dout, reverse (dout SiLU(z), C).
cudaError_t launch_heads_local(const HeadsArgs& a, const void* dout, bool bf16, cudaStream_t st);

}  // namespace sscan
