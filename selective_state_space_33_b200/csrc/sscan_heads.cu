// sscan_heads.cu -- forward of the multi-head recurrence with a P x N state per head (the
// mathematics is in sscan_heads.cuh), the segment passes that split a long sequence, and the
// one-token step.
//
// heads_walk_kernel: one block per (head, batch row, segment) walks its chunks with the state
// in the accumulators of its four warps (16 channels each), so a sequence that is not split
// is read once.  In bf16 the factors that carry fp32 quantities into a product (the state, and
// u scaled by f) go in as two bf16 parts; the entries of M are rounded to bf16 once, an error
// of the same size as the rounding of the result.
#include <cuda_runtime.h>

#include <type_traits>

#include "sscan_heads.cuh"
#include "sscan_vec.cuh"

namespace sscan {
namespace {

constexpr int kThreads = 128;

enum { kWalkOut = 0, kWalkLocal = 1, kWalkLocalRev = 2 };

template <typename T, int NT, int MODE>
struct WalkSmem {
    using Pt = HeadsPitch<T, NT>;
    static constexpr bool two = !Mma<T>::kExact32, out = MODE == kWalkOut;
    alignas(16) T x[kQ * Pt::P];                            // u (reverse: dout)
    alignas(16) T fh[kQ * Pt::P];                           // its scaled copy, and the second part
    alignas(16) T fl[two ? kQ * Pt::P : 1];
    alignas(16) T B[kQ * Pt::N];                            // B (reverse: C)
    alignas(16) T C[out ? kQ * Pt::N : 1];
    alignas(16) T sh[out ? kHeadDim * Pt::N : 1];           // the state, [p][n]
    alignas(16) T sl[out && two ? kHeadDim * Pt::N : 1];
    ChunkScalars s;
};

template <typename T, int NT, int MODE>
__global__ void __launch_bounds__(kThreads) heads_walk_kernel(HeadsArgs a, const T* dout) {
    using Pt = HeadsPitch<T, NT>;
    using M = Mma<T>;
    constexpr int NTL = NT / 8, PTL = kHeadDim / 8;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<WalkSmem<T, NT, MODE>*>(smem_raw);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int64_t b = blockIdx.y, seg = blockIdx.x / a.H;
    const int h = (int)(blockIdx.x - seg * a.H), grp = h / (a.H / a.G);
    const int64_t c0 = seg * a.seg_chunks, c1 = c0 + a.seg_chunks < a.chunks ? c0 + a.seg_chunks : a.chunks;
    const int64_t bh = b * a.H + h;
    const T *u = static_cast<const T*>(a.u), *z = static_cast<const T*>(a.z);
    const T* Bm = static_cast<const T*>(MODE == kWalkLocalRev ? a.C : a.B);

    // the state: rows p = 16 w + g and + 8, columns n = 8 j + 2 q and + 1
    float S[NTL][4];
    zero_acc(S);
    const float* first = MODE != kWalkOut ? nullptr
                         : a.nseg > 1     ? a.states + (bh * a.nseg + seg) * a.P * a.N
                         : a.h0           ? a.h0 + bh * a.P * a.N
                                          : nullptr;
    auto each_state = [&](auto&& fn) {
#pragma unroll
        for (int j = 0; j < NTL; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = 16 * w + g + (i >> 1) * 8, n = 8 * j + 2 * q + (i & 1);
                if (p < a.P && n < a.N) fn(S[j][i], (int64_t)p * a.N + n);
            }
    };
    if (first) each_state([&](float& v, int64_t at) { v = first[at]; });
    double total = 0.0;

    for (int64_t ci = 0; ci < c1 - c0; ++ci) {
        const int64_t c = MODE == kWalkLocalRev ? c1 - 1 - ci : c0 + ci;
        const int64_t t0 = c * kQ, rows = a.L - t0 < kQ ? a.L - t0 : kQ;
        const int64_t row = (b * a.L + t0) * a.H + h, rowg = (b * a.L + t0) * a.G + grp;
        __syncthreads();  // the last chunk's readers are done
        load_tile<T, kHeadDim>(sm.x, Pt::P, (MODE == kWalkLocalRev ? dout : u) + row * a.P, (int64_t)a.H * a.P, rows,
                               a.P, a.vec, tid, kThreads);
        load_tile<T, NT>(sm.B, Pt::N, Bm + rowg * a.N, (int64_t)a.G * a.N, rows, a.N, a.vec, tid, kThreads);
        if constexpr (MODE == kWalkOut) {
            load_tile<T, NT>(sm.C, Pt::N, static_cast<const T*>(a.C) + rowg * a.N, (int64_t)a.G * a.N, rows, a.N, a.vec,
                             tid, kThreads);
#pragma unroll
            for (int j = 0; j < NTL; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    split_store<T>(sm.sh, sm.sl, (16 * w + g + (i >> 1) * 8) * Pt::N + 8 * j + 2 * q + (i & 1), S[j][i]);
        }
        if (w == 0) chunk_scalars<T>(sm.s, a, b, h, t0);
        __syncthreads();
        // the scaled copy of x; in reverse the scale is exp(c_t) and SiLU(z) comes in too
        int bad = 0;
        for (int i = tid; i < kQ * kHeadDim; i += kThreads) {
            const int t = i / kHeadDim, p = i - t * kHeadDim;
            float v = to_f32<T>(sm.x[t * Pt::P + p]);
            if constexpr (MODE == kWalkLocalRev) {
                if (z && t < rows && p < a.P) v *= silu(to_f32<T>(z[(row + (int64_t)t * a.H) * a.P + p]));
                split_store<T>(sm.fh, sm.fl, t * Pt::P + p, v * sm.s.e[t]);
            } else {
                split_store<T>(sm.fh, sm.fl, t * Pt::P + p, v * sm.s.f[t]);
                if (MODE == kWalkOut && !(fabsf(v) <= 3.4e38f)) {
                    // a value that is not finite must not meet the zeros of M above the diagonal:
                    // it is left out of the product and added to its own rows below
                    bad = 1;
                    sm.x[t * Pt::P + p] = from_f32<T>(0.f);
                }
            }
        }
        if (MODE == kWalkOut) bad = __syncthreads_or(bad);
        else __syncthreads();

        if constexpr (MODE == kWalkOut) {
            float y[PTL][4];
            zero_acc(y);
            warp_gemm<T, false, false, PTL>(y, sm.C, Pt::N, 16 * w, sm.sh, Pt::N, 0, 0, NT);
            if constexpr (!M::kExact32) warp_gemm<T, false, false, PTL>(y, sm.C, Pt::N, 16 * w, sm.sl, Pt::N, 0, 0, NT);
            const int ta = 16 * w + g, tb = ta + 8;
#pragma unroll
            for (int j = 0; j < PTL; ++j) {
                y[j][0] *= sm.s.e[ta];
                y[j][1] *= sm.s.e[ta];
                y[j][2] *= sm.s.e[tb];
                y[j][3] *= sm.s.e[tb];
            }
            // M U, 16 columns s of M at a time, up to the diagonal
            for (int s0 = 0; s0 <= 16 * w; s0 += 16) {
                float m[2][4];
                zero_acc(m);
                warp_gemm<T, false, false, 2>(m, sm.C, Pt::N, 16 * w, sm.B, Pt::N, s0, 0, NT);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = ta + (i >> 1) * 8, s = s0 + 8 * j + 2 * q + (i & 1);
                        m[j][i] = s <= t ? m[j][i] * (chunk_decay(sm.s, t, s) * sm.s.w[s]) : 0.f;
                    }
#pragma unroll
                for (int k = 0; k < 2; k += M::KT) {
                    typename M::A fa;
                    M::from_acc(fa, m + k);
#pragma unroll
                    for (int j = 0; j < PTL; j += 2) {
                        typename M::B b0, b1;
                        M::load_bt2(b0, b1, sm.x, Pt::P, 8 * j, s0 + 8 * k);
                        M::mma(y[j], fa, b0);
                        M::mma(y[j + 1], fa, b1);
                    }
                }
            }
            const float D = a.D ? __ldg(a.D + h) : 0.f;
#pragma unroll
            for (int j = 0; j < PTL; ++j)
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const int t = ta + (i >> 1) * 8, p = 8 * j + 2 * q;
                    if (t >= rows) continue;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (p + k >= a.P) continue;
                        const int64_t at = (row + (int64_t)t * a.H) * a.P + p + k;
                        float v = y[j][i + k];
                        float x = to_f32<T>(sm.x[t * Pt::P + p + k]);
                        if (bad) {
                            x = to_f32<T>(u[at]);
                            for (int s = 0; s <= t; ++s) {
                                const float xs = to_f32<T>(u[(row + (int64_t)s * a.H) * a.P + p + k]);
                                if (fabsf(xs) <= 3.4e38f) continue;
                                float dot = 0.f;
                                for (int n = 0; n < a.N; ++n)
                                    dot = fmaf(to_f32<T>(sm.C[t * Pt::N + n]), to_f32<T>(sm.B[s * Pt::N + n]), dot);
                                v += dot * (chunk_decay(sm.s, t, s) * sm.s.w[s]) * xs;
                            }
                        }
                        v = a.D ? fmaf(D, x, v) : v;
                        if (z) v *= silu(to_f32<T>(z[at]));
                        static_cast<T*>(a.out)[at] = from_f32<T>(v);
                    }
                }
        }
        // S' = exp(c_end) S + (f U)^T B
        const float dec = ex2(sm.s.total * kLog2e);
        total += sm.s.total;
#pragma unroll
        for (int j = 0; j < NTL; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[j][i] *= dec;
        warp_gemm<T, true, true, NTL>(S, sm.fh, Pt::P, 16 * w, sm.B, Pt::N, 0, 0, kQ);
        if constexpr (!M::kExact32) warp_gemm<T, true, true, NTL>(S, sm.fl, Pt::P, 16 * w, sm.B, Pt::N, 0, 0, kQ);
    }
    if constexpr (MODE == kWalkOut) {
        if (a.h_last && seg == a.nseg - 1) {
            float* o = a.h_last + bh * a.P * a.N;
            each_state([&](float& v, int64_t at) { o[at] = v; });
        }
    } else {
        float* o = a.states + (bh * a.nseg + seg) * a.P * a.N;
        each_state([&](float& v, int64_t at) { o[at] = v; });
        if (tid == 0) a.decays[bh * a.nseg + seg] = (float)total;
    }
}

// Turns segment end states from zero into entering states, in place, for every (batch, head,
// state): forward from `first` (h0 or zero) in segment order, or for the adjoint from zero in
// reverse order.  The value after the last segment goes to `last`.
template <int V>
__global__ void __launch_bounds__(128) heads_carry_kernel(HeadsArgs a, bool reverse, const float* first, float* last) {
    const int64_t per = (int64_t)a.P * a.N / V;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t bh = i / per;
    if (bh >= a.batch * a.H) return;
    const int64_t at = (i - bh * per) * V, PN = (int64_t)a.P * a.N;
    float* st = a.states + bh * a.nseg * PN + at;
    const float* dec = a.decays + bh * a.nseg;
    float cur[V];
#pragma unroll
    for (int v = 0; v < V; ++v) cur[v] = first ? first[bh * PN + at + v] : 0.f;
    constexpr int kAhead = 8;
    for (int64_t k0 = 0; k0 < a.nseg; k0 += kAhead) {
        Vec<float, V> loc[kAhead];
        float d[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (k0 + k < a.nseg) {
                const int64_t s = reverse ? a.nseg - 1 - (k0 + k) : k0 + k;
                loc[k].load_rw(st + s * PN);
                d[k] = dec[s];
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (k0 + k < a.nseg) {
                const int64_t s = reverse ? a.nseg - 1 - (k0 + k) : k0 + k;
                float x[V];
                loc[k].get(x);
                store_vec<V>(st + s * PN, cur);
                const float e = ex2(d[k] * kLog2e);
#pragma unroll
                for (int v = 0; v < V; ++v) cur[v] = fmaf(e, cur[v], x[v]);
            }
    }
    if (last) {
#pragma unroll
        for (int v = 0; v < V; ++v) last[bh * PN + at + v] = cur[v];
    }
}

// One token: a warp owns `rows` channels of one (batch, head) in turn; lanes run along n.
template <typename T>
__global__ void __launch_bounds__(128) heads_step_kernel(HeadsArgs a, float* state) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t bh = unit / a.P;
    if (bh >= a.batch * a.H) return;
    const int p = (int)(unit - bh * a.P);
    const int64_t b = bh / a.H;
    const int h = (int)(bh - b * a.H);
    const int64_t bg = b * a.G + h / (a.H / a.G);
    const float A = __ldg(a.A + h);
    const float r = IO<T>::load(static_cast<const T*>(a.delta_raw), bh) + (a.bias ? __ldg(a.bias + h) : 0.f);
    const float dl = a.softplus ? (r > 20.f ? r : log1pf(expf(r))) : r;
    const float qv = dl * A, dec = ex2(qv * kLog2e);
    const float x = IO<T>::load(static_cast<const T*>(a.u), bh * a.P + p);
    const float wx = (A != 0.f ? expm1f(qv) / A : dl) * x;
    float* sp = state + (bh * a.P + p) * a.N;
    float y = 0.f;
    for (int n = lane; n < a.N; n += 32) {
        const float s = fmaf(dec, sp[n], wx * IO<T>::load(static_cast<const T*>(a.B), bg * a.N + n));
        sp[n] = s;
        y = fmaf(s, IO<T>::load(static_cast<const T*>(a.C), bg * a.N + n), y);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (lane == 0) {
        if (a.D) y = fmaf(__ldg(a.D + h), x, y);
        if (a.z) y *= silu(IO<T>::load(static_cast<const T*>(a.z), bh * a.P + p));
        IO<T>::store(static_cast<T*>(a.out), bh * a.P + p, y);
    }
}

// ---------------------------------------------------------------- host

template <typename T, int NT, int MODE>
cudaError_t walk(const HeadsArgs& a, const void* dout, cudaStream_t st) {
    auto* k = heads_walk_kernel<T, NT, MODE>;
    constexpr size_t smem = sizeof(WalkSmem<T, NT, MODE>);
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    k<<<dim3((unsigned)(a.H * a.nseg), (unsigned)a.batch), kThreads, smem, st>>>(a, static_cast<const T*>(dout));
    api_count_launch();
    return cudaGetLastError();
}

template <typename T, int MODE>
cudaError_t walk_n(const HeadsArgs& a, const void* dout, cudaStream_t st) {
    if (a.N <= 16) return walk<T, 16, MODE>(a, dout, st);
    if (a.N <= 32) return walk<T, 32, MODE>(a, dout, st);
    if (a.N <= 64) return walk<T, 64, MODE>(a, dout, st);
    return walk<T, 128, MODE>(a, dout, st);
}

// Segments of a forward pass: one block per (batch, head) where those fill the GPU, else
// enough segments for about four blocks per SM, of at least four chunks.
void plan_heads(HeadsArgs& a) {
    const int64_t bh = a.batch * a.H;
    int64_t nseg = 1;
    if (bh < 3 * 148) {
        nseg = (4 * 148 + bh - 1) / bh;
        if (nseg > (a.chunks + 3) / 4) nseg = (a.chunks + 3) / 4;
        if (nseg < 2) nseg = 1;
    }
    a.seg_chunks = (a.chunks + nseg - 1) / nseg;
    a.nseg = (a.chunks + a.seg_chunks - 1) / a.seg_chunks;
}

size_t split_bytes(const HeadsArgs& a) {
    const size_t bh = (size_t)(a.batch * a.H);
    return round256(bh * a.nseg * a.P * a.N * sizeof(float)) + round256(bh * a.nseg * sizeof(float));
}

}  // namespace

sscan_status check_heads(const sscan_heads_problem* p) {
    if (!p) return api_fail(SSCAN_ERR_INVALID_ARG, "problem is NULL");
    if (p->batch < 0 || p->seqlen < 0 || p->heads < 0)
        return api_fail(SSCAN_ERR_INVALID_ARG, "negative size (batch %lld, seqlen %lld, heads %lld)",
                        (long long)p->batch, (long long)p->seqlen, (long long)p->heads);
    if (p->headdim < 1 || p->dstate < 1 || p->groups < 1)
        return api_fail(SSCAN_ERR_INVALID_ARG, "headdim, dstate and groups must be >= 1");
    if (p->headdim > kHeadDim || p->dstate > 128)
        return api_fail(SSCAN_ERR_UNSUPPORTED, "headdim %lld > %d or dstate %lld > 128", (long long)p->headdim, kHeadDim,
                        (long long)p->dstate);
    if (p->heads % p->groups)
        return api_fail(SSCAN_ERR_INVALID_ARG, "heads %lld is not a multiple of groups %lld", (long long)p->heads,
                        (long long)p->groups);
    if (p->io_dtype != SSCAN_F32 && p->io_dtype != SSCAN_BF16)
        return api_fail(SSCAN_ERR_INVALID_ARG, "unknown io_dtype %d", (int)p->io_dtype);
    if (p->flags & ~SSCAN_DELTA_SOFTPLUS)
        return api_fail(SSCAN_ERR_INVALID_ARG, "unknown flag bits 0x%x", (unsigned)(p->flags & ~SSCAN_DELTA_SOFTPLUS));
    if (p->batch > 65535 || p->heads > (int64_t(1) << 24))
        return api_fail(SSCAN_ERR_UNSUPPORTED, "batch %lld > 65535 or heads %lld > 2^24", (long long)p->batch,
                        (long long)p->heads);
    if (p->heads > 0 && (p->seqlen + kQ - 1) / kQ > ((int64_t(1) << 31) - 1) / p->heads)
        return api_fail(SSCAN_ERR_UNSUPPORTED, "more than 2^31 (head, %d-step chunk) pairs", kQ);
    if (sscan_status s = api_elements(p->batch, p->seqlen, p->heads * p->headdim)) return s;
    return api_elements(p->batch, p->seqlen, p->groups * p->dstate);
}

HeadsArgs heads_args(const sscan_heads_problem* p, const void* u, const void* delta_raw, const float* delta_bias,
                     const float* A, const void* B, const void* C, const float* D_skip, const void* z,
                     const float* h0) {
    HeadsArgs a{};
    a.batch = p->batch, a.L = p->seqlen;
    a.H = (int)p->heads, a.P = (int)p->headdim, a.N = (int)p->dstate, a.G = (int)p->groups;
    a.softplus = (p->flags & SSCAN_DELTA_SOFTPLUS) ? 1 : 0;
    a.u = u, a.delta_raw = delta_raw, a.B = B, a.C = C, a.z = z;
    a.A = A, a.bias = delta_bias, a.D = D_skip, a.h0 = h0;
    a.chunks = (p->seqlen + kQ - 1) / kQ;
    const size_t es = p->io_dtype == SSCAN_BF16 ? 2 : 4;
    a.vec = a.P * es % 16 == 0 && a.N * es % 16 == 0 && aligned_to(u, 16) && aligned_to(B, 16) && aligned_to(C, 16);
    return a;
}

cudaError_t launch_heads_local(const HeadsArgs& a, const void* dout, bool bf16, cudaStream_t st) {
    if (bf16) return dout ? walk_n<__nv_bfloat16, kWalkLocalRev>(a, dout, st) : walk_n<__nv_bfloat16, kWalkLocal>(a, dout, st);
    return dout ? walk_n<float, kWalkLocalRev>(a, dout, st) : walk_n<float, kWalkLocal>(a, dout, st);
}

void launch_heads_carry(const HeadsArgs& a, bool reverse, const float* first, float* last, cudaStream_t st) {
    const int64_t all = a.batch * a.H * a.P * a.N;
    const bool four = (int64_t)a.P * a.N % 4 == 0;
    const unsigned blocks = (unsigned)((all / (four ? 4 : 1) + 127) / 128);
    if (four) heads_carry_kernel<4><<<blocks, 128, 0, st>>>(a, reverse, first, last);
    else heads_carry_kernel<1><<<blocks, 128, 0, st>>>(a, reverse, first, last);
    api_count_launch();
}

size_t heads_fwd_bytes(const sscan_heads_problem* p) {
    HeadsArgs a = heads_args(p, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
    plan_heads(a);
    return a.nseg > 1 ? split_bytes(a) : 0;
}

size_t heads_bwd_bytes(const sscan_heads_problem* p);

}  // namespace sscan

using namespace sscan;

extern "C" {

size_t sscan_heads_workspace_size(const sscan_heads_problem* p, int op) {
    if (check_heads(p) != SSCAN_OK || p->batch == 0 || p->seqlen == 0 || p->heads == 0) return 0;
    if (op == SSCAN_OP_FWD) return heads_fwd_bytes(p);
    if (op == SSCAN_OP_BWD) return heads_bwd_bytes(p);
    return 0;
}

sscan_status sscan_heads_fwd(const sscan_heads_problem* p, const void* u, const void* delta_raw,
                             const float* delta_bias, const float* A, const void* B, const void* C,
                             const float* D_skip, const void* z, const float* h0, void* out, float* h_last,
                             void* workspace, size_t workspace_bytes, void* stream) {
    api_begin();
    if (sscan_status s = check_heads(p)) return s;
    if (p->batch == 0 || p->heads == 0) return SSCAN_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->seqlen == 0) {
        if (!h_last) return SSCAN_OK;
        const size_t bytes = (size_t)(p->batch * p->heads * p->headdim * p->dstate) * sizeof(float);
        const cudaError_t e = h0 ? cudaMemcpyAsync(h_last, h0, bytes, cudaMemcpyDeviceToDevice, st)
                                 : cudaMemsetAsync(h_last, 0, bytes, st);
        return e == cudaSuccess ? SSCAN_OK : api_fail(SSCAN_ERR_CUDA, "copying h0 to h_last: %s", cudaGetErrorString(e));
    }
    if (!u || !delta_raw || !A || !B || !C || !out)
        return api_fail(SSCAN_ERR_INVALID_ARG, "u, delta_raw, A, B, C and out are required");
    if (sscan_status s = api_workspace(sscan_heads_workspace_size(p, SSCAN_OP_FWD), workspace, workspace_bytes)) return s;
    HeadsArgs a = heads_args(p, u, delta_raw, delta_bias, A, B, C, D_skip, z, h0);
    a.out = out, a.h_last = h_last;
    plan_heads(a);
    const bool bf16 = p->io_dtype == SSCAN_BF16;
    cudaError_t e = cudaSuccess;
    if (a.nseg > 1) {
        a.states = static_cast<float*>(workspace);
        a.decays = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                            round256((size_t)(a.batch * a.H * a.nseg * a.P * a.N) * sizeof(float)));
        e = launch_heads_local(a, nullptr, bf16, st);
        if (e != cudaSuccess) return api_fail(SSCAN_ERR_CUDA, "segment state kernel: %s", cudaGetErrorString(e));
        launch_heads_carry(a, false, h0, nullptr, st);
        if (sscan_status s = api_launched("segment carry kernel")) return s;
    }
    e = bf16 ? walk_n<__nv_bfloat16, kWalkOut>(a, nullptr, st) : walk_n<float, kWalkOut>(a, nullptr, st);
    if (e != cudaSuccess) return api_fail(SSCAN_ERR_CUDA, "heads forward kernel: %s", cudaGetErrorString(e));
    return SSCAN_OK;
}

sscan_status sscan_heads_step(const sscan_heads_problem* p, const void* u, const void* delta_raw,
                              const float* delta_bias, const float* A, const void* B, const void* C,
                              const float* D_skip, const void* z, float* state, void* out, void* stream) {
    api_begin();
    if (sscan_status s = check_heads(p)) return s;
    if (p->seqlen != 1)
        return api_fail(SSCAN_ERR_INVALID_ARG, "sscan_heads_step takes seqlen == 1, got %lld", (long long)p->seqlen);
    if (p->batch == 0 || p->heads == 0) return SSCAN_OK;
    if (!u || !delta_raw || !A || !B || !C || !state || !out)
        return api_fail(SSCAN_ERR_INVALID_ARG, "u, delta_raw, A, B, C, state and out are required");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->batch * p->heads * p->headdim > int64_t(1) << 32)
        return api_fail(SSCAN_ERR_UNSUPPORTED, "more than 2^32 (batch, head, channel) rows");
    HeadsArgs a = heads_args(p, u, delta_raw, delta_bias, A, B, C, D_skip, z, nullptr);
    a.out = out;
    const unsigned blocks = (unsigned)((a.batch * a.H * a.P + 3) / 4);
    if (p->io_dtype == SSCAN_BF16) heads_step_kernel<__nv_bfloat16><<<blocks, 128, 0, st>>>(a, state);
    else heads_step_kernel<float><<<blocks, 128, 0, st>>>(a, state);
    api_count_launch();
    return api_launched("heads step kernel");
}

}  // extern "C"
