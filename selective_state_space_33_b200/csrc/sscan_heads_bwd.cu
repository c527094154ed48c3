// sscan_heads_bwd.cu -- backward of the multi-head recurrence (forward and notation in
// sscan_heads.cuh).  With dy = dout SiLU(z), R the adjoint of the state leaving a chunk and S
// the state entering it, both known from the segment passes with one segment per chunk, a
// chunk's gradients are again matrix products.  With H_ts = dy_t . u_s, G_ts = C_t . B_s,
// E_ts = exp(c_t - c_s) for s <= t (0 above), M1 = G E w_s, M2 = H E w_s, d_s = exp(c_end - c_s),
// f_s = d_s w_s and e_t = exp(c_t):
//   du_s = sum_t M1_ts dy_t + f_s R B_s + D dy_s
//   dB_s = sum_t M2_ts C_t  + f_s R^T u_s        dC_t = sum_s M2_ts B_s + e_t S^T dy_t
//     (summed over the heads of a group; they share B and C, so M2 is summed first)
//   dz_t = dout_t y_t SiLU'(z_t),                y_t = sum_s M1_ts u_s + e_t S C_t + D u_t
//   dc_t = sum_s G H E w_s (row t) - w_t sum_t' G H E (column t) + e_t dy_t . S C_t
//          - w_t d_t u_t . R B_t,  and at the last step + sum_s w_s d_s u_s . R B_s + e_end R . S
//   dq_t = sum_{t' >= t} dc_t',   dw_t = sum_t' G H E (column t) + d_t u_t . R B_t
//   ddelta = dq A + dw exp(q),    dA = sum dq delta + dw dw/dA.
// A block takes one chunk of one batch row and a share of the heads of a group; dB and dC are
// accumulated over its heads in registers.  dA and ddelta_bias are fp32 sums over the whole
// sequence of differences that nearly cancel (with two bf16 parts, 16 bits, a bias gradient came out
// 8e-5 off where the same sums in fp32 lose 1e-6), so everything that feeds them (H, S C, R B)
// takes its inexact factor as three bf16 parts, 24 bits; M1 and the factors of the products
// that end in bf16 are rounded once.
// 8 x 2048, 24 heads of 64 channels, 64 states, bf16 with gate: 480 us; two blocks of eight warps per SM,
// issue slots about a third busy, the rest the latency of nine products that follow one another, and of what
// 128 registers per thread do not hold (528 bytes of spills; sixteen warps of 64 registers were tried and were slower).
#include <cuda_runtime.h>

#include "sscan_heads.cuh"
#include "sscan_plan.h"
#include "sscan_rowsum.cuh"
#include "sscan_vec.cuh"

namespace sscan {

size_t heads_bwd_bytes(const sscan_heads_problem* p);

namespace {

constexpr int kThreads = 256;

struct HeadsBwdArgs {
    HeadsArgs f;            // inputs; f.states, f.decays: S entering each chunk
    const float* R;         // [batch][H][chunks][P][N]: adjoint of the state leaving each chunk
    const void* dout;
    void *du, *ddelta, *dB, *dC, *dz;
    float* part;            // [batch * chunks][3][H]: dA, ddelta_bias, dD over the chunk
    float* bc;              // [splits][2][batch][L][G][N] partial dB, dC, or null with one split
    int splits, per_split;  // heads of a group per block
};

template <typename T, int NT>
struct BwdSmem {
    using Pt = HeadsPitch<T, NT>;
    static constexpr bool two = !Mma<T>::kExact32;
    alignas(16) T x[kQ * Pt::P];
    alignas(16) T dyh[kQ * Pt::P];
    alignas(16) T dyl[two ? kQ * Pt::P : 1];
    alignas(16) T B[kQ * Pt::N];
    alignas(16) T C[kQ * Pt::N];
    alignas(16) T sh[kHeadDim * Pt::N];          // S, [p][n]
    alignas(16) T sl[two ? kHeadDim * Pt::N : 1];
    alignas(16) T rh[kHeadDim * Pt::N];          // R, [p][n]
    alignas(16) T rl[two ? kHeadDim * Pt::N : 1];
    alignas(16) T dy3[two ? kQ * Pt::P : 8];     // third part of dy
    // M1, and at the end M2, [t][s]; before them, in bf16, the third parts of R and S
    static constexpr int M = two && Pt::N > Pt::Q ? kHeadDim * Pt::N : kQ * Pt::Q;
    alignas(16) T m1[M];
    alignas(16) T m2[M];
    ChunkScalars s;
    ChunkSteps steps;
    float row[2][kQ], col[4][kQ], qs[2][kQ], rs[2][kQ];
    float sum[2][kThreads / 32];
};

// (q e^q - expm1(q)) / q^2 = sum_k (k + 1) q^k / (k + 2)!: dw/dA = delta^2 times this.  The
// difference cancels near 0; below |q| = 1/2 the series to q^6 leaves out 2e-7.
__device__ __forceinline__ float dw_slope(float q) {
    if (fabsf(q) < 0.5f) {
        float s = 1.f / 5760.f;
        s = fmaf(s, q, 1.f / 840.f);
        s = fmaf(s, q, 1.f / 144.f);
        s = fmaf(s, q, 1.f / 30.f);
        s = fmaf(s, q, 1.f / 8.f);
        s = fmaf(s, q, 1.f / 3.f);
        return fmaf(s, q, 0.5f);
    }
    return (q * expf(q) - expm1f(q)) / (q * q);
}

__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Loads the P x N fp32 state at `at` of `states` (of `extent` elements) into its parts, tiles of T ([p][n], zero-padded).
template <typename T, int NT, typename Each>
__device__ __forceinline__ void load_state(T* hi, T* lo, T* third, const float* states, int64_t at, int64_t extent, int P, int N,
                                           int tid, Each each) {
    constexpr int pitch = HeadsPitch<T, NT>::N;
    for (int i = tid; i < kHeadDim * NT / 4; i += kThreads) {
        const int p = i / (NT / 4), n = (i - p * (NT / 4)) * 4;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (p < P && n < N) {
            const float* s = states + at + (int64_t)p * N + n;
            const int64_t i0 = at + (int64_t)p * N + n;
            if (N % 4 == 0) {
                if (in_range(i0, extent, 4)) {
                    const float4 f = __ldg(reinterpret_cast<const float4*>(s));
                    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (n + k < N && in_range(i0 + k, extent)) v[k] = __ldg(s + k);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
            const uint32_t t = split_store2<T>(hi, lo, p * pitch + n + k, v[k], v[k + 1]);
            if constexpr (!Mma<T>::kExact32) *reinterpret_cast<uint32_t*>(third + p * pitch + n + k) = t;
        }
        each(i, v);
    }
}

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, !Mma<T>::kExact32 && NT <= 64 ? 2 : 1) heads_bwd_kernel(HeadsBwdArgs k) {
    using Pt = HeadsPitch<T, NT>;
    using M = Mma<T>;
    constexpr int NTL = NT / 8, HTL = NTL > 8 ? 8 : NTL;  // dB / dC columns in passes of at most 64
    extern __shared__ __align__(16) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<BwdSmem<T, NT>*>(smem_raw);
    const HeadsArgs& a = k.f;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int wr = w & 3, wc = w >> 2;                    // 16 rows, one half of the columns
    const int ra = 16 * wr + g, rb = ra + 8, cb = 32 * wc + 2 * q;
    const int64_t b = blockIdx.y, c = blockIdx.x;
    const int grp = blockIdx.z / k.splits, split = blockIdx.z - grp * k.splits;
    const int hg = a.H / a.G, h_begin = grp * hg + split * k.per_split;
    const int h_end = (split + 1) * k.per_split < hg ? h_begin + k.per_split : (grp + 1) * hg;
    const int64_t t0 = c * kQ, rows = a.L - t0 < kQ ? a.L - t0 : kQ;
    const int64_t tok = b * a.L + t0;                     // first token of the chunk
    const T *u = static_cast<const T*>(a.u), *z = static_cast<const T*>(a.z), *dout = static_cast<const T*>(k.dout);

    load_tile<T, NT>(sm.B, Pt::N, static_cast<const T*>(a.B) + (tok * a.G + grp) * a.N, (int64_t)a.G * a.N, rows, a.N,
                     a.vec, tid, kThreads);
    load_tile<T, NT>(sm.C, Pt::N, static_cast<const T*>(a.C) + (tok * a.G + grp) * a.N, (int64_t)a.G * a.N, rows, a.N,
                     a.vec, tid, kThreads);
    __syncthreads();
    const bool lower = 32 * wc <= 16 * wr + 15;           // this warp's part of a Q x Q matrix is not all above the diagonal
    float G[4][4];
    zero_acc(G);
    if (lower) warp_gemm<T, false, false, 4>(G, sm.C, Pt::N, 16 * wr, sm.B, Pt::N, 32 * wc, 0, NT);
    float bc[NTL][4];                                     // wc = 0: dC (rows t), wc = 1: dB (rows s)
    zero_acc(bc);
    float M2[4][4];                                       // sum of M2 over the heads, which share B and C
    zero_acc(M2);

    for (int h = h_begin; h < h_end; ++h) {
        const int64_t bh = b * a.H + h;
        const float D = head_param(a, a.D, h);
        if (w == 0) chunk_scalars<T>(sm.s, a, b, h, t0, &sm.steps);
        // u, dy and their product's sum
        float dsum = 0.f, ssum = 0.f;
        constexpr int VE = 16 / sizeof(T), PER = kHeadDim / VE, LOADS = kQ * PER / kThreads;
        {
#pragma unroll
            for (int n = 0; n < LOADS; ++n) {
                const int i = tid + n * kThreads, t = i / PER, p = (i - t * PER) * VE;
                const int64_t at = ((tok + t) * a.H + h) * a.P + p;
                float xv[VE], dv[VE], zv[VE];
                if (t < rows && p < a.P && a.vec) {
                    load_vec<VE>(u + at, xv);
                    load_vec<VE>(dout + at, dv);
                    if (z) load_vec<VE>(z + at, zv);
                } else {
#pragma unroll
                    for (int j = 0; j < VE; ++j) {
                        const bool in = t < rows && p + j < a.P;
                        xv[j] = in ? IO<T>::load(u, at + j) : 0.f;
                        dv[j] = in ? IO<T>::load(dout, at + j) : 0.f;
                        if (z) zv[j] = in ? IO<T>::load(z, at + j) : 0.f;
                    }
                }
#pragma unroll
                for (int j = 0; j < VE; j += 2) {
                    if (z) dv[j] *= silu(zv[j]), dv[j + 1] *= silu(zv[j + 1]);
                    dsum = fmaf(dv[j], xv[j], fmaf(dv[j + 1], xv[j + 1], dsum));
                    const uint32_t third = split_store2<T>(sm.dyh, sm.dyl, t * Pt::P + p + j, dv[j], dv[j + 1]);
                    if constexpr (!M::kExact32) *reinterpret_cast<uint32_t*>(sm.dy3 + t * Pt::P + p + j) = third;
                }
                store_vec<VE>(sm.x + t * Pt::P + p, xv);
            }
        }
        // S then R; a thread reads the same elements of both, so their product is summed on the way
        {
            const int64_t at = (bh * a.chunks + c) * a.P * a.N;
            constexpr int PER = kHeadDim * NT / 4 / kThreads;
            float sv[PER][4];
            load_state<T, NT>(sm.sh, sm.sl, sm.m2, a.states, at, states_extent(a), a.P, a.N, tid, [&](int i, const float (&v)[4]) {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (i == tid + j * kThreads)
                        for (int e = 0; e < 4; ++e) sv[j][e] = v[e];
            });
            load_state<T, NT>(sm.rh, sm.rl, sm.m1, k.R, at, states_extent(a), a.P, a.N, tid, [&](int i, const float (&v)[4]) {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (i == tid + j * kThreads)
                        for (int e = 0; e < 4; ++e) ssum = fmaf(sv[j][e], v[e], ssum);
            });
        }
        // the next head's tiles on their way to L2 while this one is worked on
        if (h + 1 < h_end) {
            if (tid < kQ && tid < rows) {
                const int64_t at = ((tok + tid) * a.H + h + 1) * a.P;
                prefetch_l2(u + at);
                prefetch_l2(dout + at);
                if (z) prefetch_l2(z + at);
            }
            const int64_t at = ((bh + 1) * a.chunks + c) * a.P * a.N;
            for (int i = tid * 32; i < a.P * a.N; i += kThreads * 32) {
                prefetch_l2(a.states + at + i);
                prefetch_l2(k.R + at + i);
            }
        }
        dsum = warp_sum(dsum);
        ssum = warp_sum(ssum);
        if (lane == 0) sm.sum[0][w] = dsum, sm.sum[1][w] = ssum;
        __syncthreads();

        // A warp's 16 rows by 32 columns of du or dz, by way of its own part of dyl (read before) to
        // 16-byte stores; fp32 has no dyl and stores its pairs.
        auto store_part = [&](T* out, const float (&v)[4][4]) {
            if (!M::kExact32 && a.vec) {
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float lo[2] = {v[j][0], v[j][1]}, hi[2] = {v[j][2], v[j][3]};
                    store_vec<2>(sm.dyl + ra * Pt::P + cb + 8 * j, lo);
                    store_vec<2>(sm.dyl + rb * Pt::P + cb + 8 * j, hi);
                }
                __syncwarp();
                constexpr int VE = 16 / sizeof(T), PER = 32 / VE;
#pragma unroll
                for (int i = lane; i < 16 * PER; i += 32) {
                    const int t = 16 * wr + i / PER, p = 32 * wc + (i % PER) * VE;
                    if (t < rows && p < a.P)
                        *reinterpret_cast<uint4*>(out + ((tok + t) * a.H + h) * a.P + p) =
                            *reinterpret_cast<const uint4*>(sm.dyl + t * Pt::P + p);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = i < 2 ? ra : rb, p = cb + 8 * j + (i & 1);
                        if (t < rows && p < a.P) out[((tok + t) * a.H + h) * a.P + p] = from_f32<T>(v[j][i]);
                    }
            }
        };

        // H, M1 and M2, and the sums of G H E over rows and columns
        Vec<T, 2> m1v[4][2];
        float Hm[4][4];
        zero_acc(Hm);
        if (lower) {
            warp_gemm<T, false, false, 4>(Hm, sm.dyh, Pt::P, 16 * wr, sm.x, Pt::P, 32 * wc, 0, kHeadDim);
            if (!M::kExact32 && z) {
                warp_gemm<T, false, false, 4>(Hm, sm.dyl, Pt::P, 16 * wr, sm.x, Pt::P, 32 * wc, 0, kHeadDim);
                warp_gemm<T, false, false, 4>(Hm, sm.dy3, Pt::P, 16 * wr, sm.x, Pt::P, 32 * wc, 0, kHeadDim);
            }
        }
        float rowa = 0.f, rowb = 0.f;
        const float cha = sm.s.ch[ra], cla = sm.s.cl[ra], chb = sm.s.ch[rb], clb = sm.s.cl[rb];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int s0 = cb + 8 * j;
            const float2 ws = *reinterpret_cast<const float2*>(sm.s.w + s0);
            const float2 chs = *reinterpret_cast<const float2*>(sm.s.ch + s0);
            const float2 cls = *reinterpret_cast<const float2*>(sm.s.cl + s0);
            float cols[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const int t = i ? rb : ra;
                float m1[2];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float E = ex2(((i ? chb : cha) - (n ? chs.y : chs.x)) + ((i ? clb : cla) - (n ? cls.y : cls.x)));
                    const float w_ = n ? ws.y : ws.x;
                    const bool in = s0 + n <= t;
                    const float ge = in ? G[j][i + n] * E : 0.f, he = in ? Hm[j][i + n] * E : 0.f;
                    const float pair = in ? ge * Hm[j][i + n] : 0.f;
                    cols[n] += pair;
                    (i ? rowb : rowa) += pair * w_;
                    m1[n] = ge * w_;
                    M2[j][i + n] = fmaf(he, w_, M2[j][i + n]);
                }
                m1v[j][i / 2].set(m1);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v = cols[i];
#pragma unroll
                for (int o = 4; o < 32; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (g == 0) sm.col[wr][s0 + i] = v;
            }
        }
        rowa = quad_sum(rowa);
        rowb = quad_sum(rowb);
        if (q == 0) sm.row[wc][ra] = rowa, sm.row[wc][rb] = rowb;
        // R B (rows s, columns p) and S C (rows t, columns p): both end in fp32 sums over the sequence
        // that nearly cancel, so R, S and dy enter with 24 bits
        float x[4][4], y[4][4];
        {
            zero_acc(x);
            warp_gemm<T, false, false, 4>(x, sm.B, Pt::N, 16 * wr, sm.rh, Pt::N, 32 * wc, 0, NT);
            if constexpr (!M::kExact32) {
                warp_gemm<T, false, false, 4>(x, sm.B, Pt::N, 16 * wr, sm.rl, Pt::N, 32 * wc, 0, NT);
                warp_gemm<T, false, false, 4>(x, sm.B, Pt::N, 16 * wr, sm.m1, Pt::N, 32 * wc, 0, NT);
            }
            float va = 0.f, vb = 0.f;
            const float fa = sm.s.f[ra], fb = sm.s.f[rb];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float u0[2], u1[2];
                load_shared<2>(sm.x + ra * Pt::P + cb + 8 * j, u0);
                load_shared<2>(sm.x + rb * Pt::P + cb + 8 * j, u1);
                va = fmaf(x[j][0], u0[0], fmaf(x[j][1], u0[1], va));
                vb = fmaf(x[j][2], u1[0], fmaf(x[j][3], u1[1], vb));
                x[j][0] *= fa, x[j][1] *= fa;
                x[j][2] *= fb, x[j][3] *= fb;
            }
            va = quad_sum(va);
            vb = quad_sum(vb);
            if (q == 0) sm.rs[wc][ra] = va, sm.rs[wc][rb] = vb;
        }
        {
            zero_acc(y);
            warp_gemm<T, false, false, 4>(y, sm.C, Pt::N, 16 * wr, sm.sh, Pt::N, 32 * wc, 0, NT);
            if constexpr (!M::kExact32) {
                warp_gemm<T, false, false, 4>(y, sm.C, Pt::N, 16 * wr, sm.sl, Pt::N, 32 * wc, 0, NT);
                warp_gemm<T, false, false, 4>(y, sm.C, Pt::N, 16 * wr, sm.m2, Pt::N, 32 * wc, 0, NT);
            }
            const float ea = sm.s.e[ra], eb = sm.s.e[rb];
            float va = 0.f, vb = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const int at = (i ? rb : ra) * Pt::P + cb + 8 * j;
                    float dy[2];
                    load_shared<2>(sm.dyh + at, dy);
                    if constexpr (!M::kExact32) {
                        float lo[2];
                        load_shared<2>(sm.dyl + at, lo);
                        dy[0] += lo[0], dy[1] += lo[1];
                        if (z) {
                            load_shared<2>(sm.dy3 + at, lo);
                            dy[0] += lo[0], dy[1] += lo[1];
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        y[j][i + n] *= i ? eb : ea;
                        (i ? vb : va) += y[j][i + n] * dy[n];
                        x[j][i + n] = fmaf(D, dy[n], x[j][i + n]);
                    }
                }
            va = quad_sum(va);
            vb = quad_sum(vb);
            if (q == 0) sm.qs[wc][ra] = va, sm.qs[wc][rb] = vb;
        }
        if constexpr (!M::kExact32) __syncthreads();  // the third parts, whose place M1 takes, are read
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m1v[j][0].store(sm.m1 + ra * Pt::Q + cb + 8 * j);
            m1v[j][1].store(sm.m1 + rb * Pt::Q + cb + 8 * j);
        }
        __syncthreads();

        // du, and with a gate dz
        {
            warp_gemm<T, true, true, 4>(x, sm.m1, Pt::Q, 16 * wr, sm.dyh, Pt::P, 32 * wc, 16 * wr, kQ);
            store_part(static_cast<T*>(k.du), x);
            if (z) {
                // dout and z again, in this warp's layout, ahead of the product that hides their latency
                Vec<T, 2> dv[4][2], zv[4][2];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int t = i ? rb : ra, p = cb + 8 * j;
                        const int64_t at = ((tok + t) * a.H + h) * a.P + p;
                        dv[j][i].zero();
                        zv[j][i].zero();
                        if (t < rows && p < a.P) {
                            if (a.vec) {
                                dv[j][i].load(dout + at);
                                zv[j][i].load(z + at);
                            } else {
                                const bool two = p + 1 < a.P;
                                const float d2[2] = {IO<T>::load(dout, at), two ? IO<T>::load(dout, at + 1) : 0.f};
                                const float z2[2] = {IO<T>::load(z, at), two ? IO<T>::load(z, at + 1) : 0.f};
                                dv[j][i].set(d2);
                                zv[j][i].set(z2);
                            }
                        }
                    }
                warp_gemm<T, false, true, 4>(y, sm.m1, Pt::Q, 16 * wr, sm.x, Pt::P, 32 * wc, 0, 16 * wr + 16);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float uv[2], d2[2], z2[2];
                        load_shared<2>(sm.x + (i ? rb : ra) * Pt::P + cb + 8 * j, uv);
                        dv[j][i].get(d2);
                        zv[j][i].get(z2);
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            y[j][2 * i + n] = d2[n] * fmaf(D, uv[n], y[j][2 * i + n]) * dsilu(z2[n]);
                    }
                store_part(static_cast<T*>(k.dz), y);
            }
        }
        // dC (wc = 0, rows t) or dB (wc = 1, rows s), at most 64 columns n at a time
#pragma unroll
        for (int n0 = 0; n0 < NTL; n0 += HTL) {
            float v[HTL][4];
            zero_acc(v);
            if (wc == 0) warp_gemm<T, false, true, HTL>(v, sm.dyh, Pt::P, 16 * wr, sm.sh, Pt::N, 8 * n0, 0, kHeadDim);
            // with a gate dy is rounded too: the second part of S keeps dC to one more rounding, as dB
            if (!M::kExact32 && z && wc == 0)
                warp_gemm<T, false, true, HTL>(v, sm.dyh, Pt::P, 16 * wr, sm.sl, Pt::N, 8 * n0, 0, kHeadDim);
            if (wc != 0) warp_gemm<T, false, true, HTL>(v, sm.x, Pt::P, 16 * wr, sm.rh, Pt::N, 8 * n0, 0, kHeadDim);
            const float fa = wc == 0 ? sm.s.e[ra] : sm.s.f[ra], fb = wc == 0 ? sm.s.e[rb] : sm.s.f[rb];
#pragma unroll
            for (int j = 0; j < HTL; ++j) {
                v[j][0] *= fa, v[j][1] *= fa;
                v[j][2] *= fb, v[j][3] *= fb;
            }
#pragma unroll
            for (int j = 0; j < HTL; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) bc[n0 + j][i] += v[j][i];
        }
        __syncthreads();
        // the scalars' gradients: one warp, steps 2 lane and 2 lane + 1
        if (w == 0) {
            const float A = head_param(a, a.A, h), end = ex2(sm.s.total * kLog2e);
            float ss = 0.f, ds = 0.f;
#pragma unroll
            for (int i = 0; i < kThreads / 32; ++i) ds += sm.sum[0][i], ss += sm.sum[1][i];
            double dc[2];
            float dw[2], tail = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                const float col = (sm.col[0][t] + sm.col[1][t]) + (sm.col[2][t] + sm.col[3][t]);
                const float rb_ = sm.s.d[t] * (sm.rs[0][t] + sm.rs[1][t]), wt = sm.s.w[t];
                dw[i] = col + rb_;
                tail = fmaf(wt, rb_, tail);
                dc[i] = (double)(sm.row[0][t] + sm.row[1][t]) + (double)(sm.qs[0][t] + sm.qs[1][t]) - (double)wt * dw[i];
            }
            const double last = (double)warp_sum(tail) + (double)end * ss;
            double run = dc[0] + dc[1];
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const double v = __shfl_down_sync(0xffffffffu, run, o);
                if (lane + o < 32) run += v;
            }
            const double dq2[2] = {run + last, run - dc[0] + last};
            float sa = 0.f, sb = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                if (t >= rows) continue;
                const float dl = sm.steps.dl[t], qv = dl * A;
                // dq_t is e^q_t R . S, got as a difference of sums that are not small with it; below
                // q = -20 it is under 2^-28 of R . S, less than those sums' roundings, which a large
                // step size would magnify
                const float dq = qv < -20.f ? 0.f : (float)dq2[i];
                float r = fmaf(dq, A, dw[i] * ex2(qv * kLog2e));
                if (a.softplus) r *= sigmoid(sm.steps.raw[t]);
                sa += fmaf(dq, dl, dw[i] * dl * dl * dw_slope(qv));
                sb += r;
                IO<T>::store(static_cast<T*>(k.ddelta), (tok + t) * a.H + h, r);
            }
            sa = warp_sum(sa);
            sb = warp_sum(sb);
            if (lane == 0) {
                const int64_t at = (b * a.chunks + c) * 3 * a.H + h, extent = a.batch * a.chunks * 3 * a.H;
                float* o = k.part + at;
                if (in_range(at, extent)) o[0] = sa;
                if (in_range(at + a.H, extent)) o[a.H] = sb;
                if (in_range(at + 2 * a.H, extent)) o[2 * a.H] = ds;
            }
        }
        __syncthreads();
    }
    // M2 B and M2^T C, once for all heads, M2 in two parts
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        split_store2<T>(sm.m1, sm.m2, ra * Pt::Q + cb + 8 * j, M2[j][0], M2[j][1]);
        split_store2<T>(sm.m1, sm.m2, rb * Pt::Q + cb + 8 * j, M2[j][2], M2[j][3]);
    }
    __syncthreads();
    auto through_m2 = [&](const T* m) {
        if (wc == 0) warp_gemm<T, false, true, NTL>(bc, m, Pt::Q, 16 * wr, sm.B, Pt::N, 0, 0, 16 * wr + 16);
        else warp_gemm<T, true, true, NTL>(bc, m, Pt::Q, 16 * wr, sm.C, Pt::N, 0, 16 * wr, kQ);
    };
    through_m2(sm.m1);
    if constexpr (!M::kExact32) through_m2(sm.m2);
    // dC or dB over this block's heads
#pragma unroll
    for (int j = 0; j < NTL; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = i < 2 ? ra : rb, n = 8 * j + 2 * q + (i & 1);
            if (t >= rows || n >= a.N) continue;
            const int64_t at = ((tok + t) * a.G + grp) * a.N + n;
            if (k.bc) {
                const int64_t n_bc = a.batch * a.L * a.G * a.N, to = (2 * (int64_t)split + wc) * n_bc + at;
                if (in_range(to, 2 * k.splits * n_bc)) k.bc[to] = bc[j][i];
            } else static_cast<T*>(wc == 0 ? k.dC : k.dB)[at] = from_f32<T>(bc[j][i]);
        }
}

// dB and dC from the splits' partial sums, in order.
template <typename T>
__global__ void __launch_bounds__(256) heads_bc_kernel(const float* bc, T* dB, T* dC, int64_t n, int splits) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= 2 * n) return;
    float s = 0.f;
    for (int k = 0; k < splits; ++k) s += in_range(2 * k * n + i, 2 * splits * n) ? __ldg(bc + 2 * k * n + i) : 0.f;
    if (i < n) dC[i] = from_f32<T>(s);
    else dB[i - n] = from_f32<T>(s);
}

// Partial rows are [3][H]: dA, ddelta_bias, dD.
struct HeadsGradPut {
    float *dA, *dbias, *dD;
    int64_t H;
    __device__ void operator()(int64_t c, float s) const {
        const int64_t k = c / H, h = c - k * H;
        float* to = k == 0 ? dA : k == 1 ? dbias : dD;
        if (to && in_range(h, H)) to[h] = s;
    }
};

// ---------------------------------------------------------------- host

template <typename T, int NT>
cudaError_t bwd(const HeadsBwdArgs& k, cudaStream_t st) {
    auto* fn = heads_bwd_kernel<T, NT>;
    constexpr size_t smem = sizeof(BwdSmem<T, NT>);
    static_assert(smem <= 227 * 1024, "the tiles of one chunk must fit a block's shared memory");
    static_assert(sizeof(T) == 4 || NT > 64 || 2 * (smem + 1024) <= 228 * 1024, "two blocks per SM up to 64 states");
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    fn<<<dim3((unsigned)k.f.chunks, (unsigned)k.f.batch, (unsigned)(k.f.G * k.splits)), kThreads, smem, st>>>(k);
    api_count_launch();
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_n(const HeadsBwdArgs& k, cudaStream_t st) {
    if (k.f.N <= 16) return bwd<T, 16>(k, st);
    if (k.f.N <= 32) return bwd<T, 32>(k, st);
    if (k.f.N <= 64) return bwd<T, 64>(k, st);
    return bwd<T, 128>(k, st);
}

// Blocks per (chunk, batch row, group): the heads of a group are shared among enough blocks
// for about four per SM.
void plan_splits(const sscan_heads_problem* p, int64_t chunks, int* splits, int* per) {
    const int64_t hg = p->heads / p->groups, base = chunks * p->batch * p->groups;
    int64_t n = (4 * kSmCount + base - 1) / base;
    if (n > hg) n = hg;
    const int64_t each = (hg + n - 1) / n;
    *per = (int)each;
    *splits = (int)((hg + each - 1) / each);
}

struct BwdLayout {
    size_t S, R, dec, part, bc, bytes;
    int splits, per;
};

BwdLayout bwd_layout(const sscan_heads_problem* p) {
    BwdLayout l{};
    const int64_t chunks = (p->seqlen + kQ - 1) / kQ;
    const size_t bhc = (size_t)(p->batch * p->heads * chunks);
    const size_t state = round256(bhc * p->headdim * p->dstate * sizeof(float));
    plan_splits(p, chunks, &l.splits, &l.per);
    l.S = 0;
    l.R = state;
    l.dec = 2 * state;
    l.part = l.dec + round256(bhc * sizeof(float));
    l.bc = l.part + round256((size_t)(p->batch * chunks * 3 * p->heads) * sizeof(float));
    l.bytes = l.bc + (l.splits > 1 ? round256((size_t)l.splits * 2 * p->batch * p->seqlen * p->groups * p->dstate * sizeof(float)) : 0);
    return l;
}

}  // namespace

size_t heads_bwd_bytes(const sscan_heads_problem* p) { return bwd_layout(p).bytes; }

}  // namespace sscan

using namespace sscan;

extern "C" sscan_status sscan_heads_bwd(const sscan_heads_problem* p, const void* u, const void* delta_raw,
                                        const float* delta_bias, const float* A, const void* B, const void* C,
                                        const float* D_skip, const void* z, const float* h0, const void* dout,
                                        void* du, void* ddelta_raw, float* ddelta_bias, float* dA, void* dB, void* dC,
                                        float* dD, void* dz, float* dh0, void* workspace, size_t workspace_bytes,
                                        void* stream) {
    api_begin();
    if (sscan_status s = check_heads(p)) return s;
    if ((z == nullptr) != (dz == nullptr)) return api_fail(SSCAN_ERR_INVALID_ARG, "dz must be given exactly when z is");
    if (dD && !D_skip) return api_fail(SSCAN_ERR_INVALID_ARG, "dD needs D_skip");
    if (ddelta_bias && !delta_bias) return api_fail(SSCAN_ERR_INVALID_ARG, "ddelta_bias needs delta_bias");
    if (p->heads > 0 && !dA) return api_fail(SSCAN_ERR_INVALID_ARG, "dA is required");
    const bool bf16 = p->io_dtype == SSCAN_BF16;
    const size_t es = bf16 ? 2 : 4;
    const int64_t state = p->batch * p->heads * p->headdim * p->dstate;
    const int64_t tokens = p->batch * p->seqlen, bcn = tokens * p->groups * p->dstate;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (tokens == 0 || p->heads == 0) {  // sums over nothing
        cudaError_t e = cudaSuccess;
        for (float* o : {dA, ddelta_bias, dD})
            if (e == cudaSuccess && o && p->heads) e = cudaMemsetAsync(o, 0, (size_t)p->heads * sizeof(float), st);
        if (e == cudaSuccess && dh0 && state) e = cudaMemsetAsync(dh0, 0, (size_t)state * sizeof(float), st);
        for (void* o : {dB, dC})
            if (e == cudaSuccess && o && bcn) e = cudaMemsetAsync(o, 0, (size_t)bcn * es, st);
        return e == cudaSuccess ? SSCAN_OK : api_fail(SSCAN_ERR_CUDA, "zeroing gradients: %s", cudaGetErrorString(e));
    }
    if (!u || !delta_raw || !A || !B || !C || !dout || !du || !ddelta_raw || !dB || !dC)
        return api_fail(SSCAN_ERR_INVALID_ARG, "u, delta_raw, A, B, C, dout, du, ddelta_raw, dB and dC are required");
    const BwdLayout l = bwd_layout(p);
    if ((int64_t)p->groups * l.splits > 65535)
        return api_fail(SSCAN_ERR_UNSUPPORTED, "more than 65535 (group, head share) blocks");
    if (sscan_status s = api_workspace(l.bytes, workspace, workspace_bytes)) return s;
    char* ws = static_cast<char*>(workspace);
    HeadsBwdArgs k{};
    HeadsArgs& a = k.f;
    a = heads_args(p, u, delta_raw, delta_bias, A, B, C, D_skip, z, h0);
    a.vec = a.vec && aligned_to(z, 16) && aligned_to(dout, 16) && aligned_to(du, 16) && aligned_to(dz, 16);
    a.nseg = a.chunks;
    a.seg_chunks = 1;
    a.decays = reinterpret_cast<float*>(ws + l.dec);
    // S entering each chunk
    a.states = reinterpret_cast<float*>(ws + l.S);
    cudaError_t e = launch_heads_local(a, nullptr, bf16, st);
    if (e != cudaSuccess) return api_fail(SSCAN_ERR_CUDA, "chunk state kernel: %s", cudaGetErrorString(e));
    launch_heads_carry(a, false, h0, nullptr, st);
    // R leaving each chunk; past the first it is the adjoint of h0
    HeadsArgs r = a;
    r.states = reinterpret_cast<float*>(ws + l.R);
    e = launch_heads_local(r, dout, bf16, st);
    if (e != cudaSuccess) return api_fail(SSCAN_ERR_CUDA, "chunk adjoint kernel: %s", cudaGetErrorString(e));
    launch_heads_carry(r, true, nullptr, dh0, st);
    if (sscan_status s = api_launched("chunk carry kernels")) return s;
    k.R = r.states;
    k.dout = dout, k.du = du, k.ddelta = ddelta_raw, k.dB = dB, k.dC = dC, k.dz = dz;
    k.part = reinterpret_cast<float*>(ws + l.part);
    k.splits = l.splits, k.per_split = l.per;
    k.bc = l.splits > 1 ? reinterpret_cast<float*>(ws + l.bc) : nullptr;
    e = bf16 ? bwd_n<__nv_bfloat16>(k, st) : bwd_n<float>(k, st);
    if (e != cudaSuccess) return api_fail(SSCAN_ERR_CUDA, "heads backward kernel: %s", cudaGetErrorString(e));
    if (k.bc) {
        const unsigned blocks = (unsigned)((2 * bcn + 255) / 256);
        if (bf16) heads_bc_kernel<<<blocks, 256, 0, st>>>(k.bc, static_cast<__nv_bfloat16*>(dB), static_cast<__nv_bfloat16*>(dC), bcn, l.splits);
        else heads_bc_kernel<<<blocks, 256, 0, st>>>(k.bc, static_cast<float*>(dB), static_cast<float*>(dC), bcn, l.splits);
        api_count_launch();
    }
    launch_rowsum(k.part, p->batch * a.chunks, 3 * p->heads, HeadsGradPut{dA, ddelta_bias, dD, p->heads}, st);
    api_count_launch();
    return api_launched("heads gradient sums");
}
