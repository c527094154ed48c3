// sscan_heads.cu -- forward of the multi-head recurrence with a P x N state per head (the
// mathematics is in sscan_heads.cuh), the segment passes that split a long sequence, and the
// one-token step.
//
// heads_walk_kernel: one block per (head, batch row, segment) walks its chunks with the state
// in the accumulators of its warps, so a sequence that is not split is read once.  The next
// chunk's tiles arrive by cp.async, and a warp of its own works out the next chunk's
// scalars (exponentials and a running sum in fp64: a long chain of dependent operations),
// while the other warps run the products of this chunk.  In bf16 the factor that carries an
// fp32 quantity into the state (u or B scaled by f) goes in as three bf16 parts, the state
// read by the outputs as two, and the entries of M are rounded to bf16 once, an error of the
// same size as the rounding of the result.
// 8 x 2048, 80 heads of 64 channels, 16 states, bf16 with gate: 243 us (508 MB, 2.1 TB/s); issue
// slots 54% busy with three blocks per SM, no pipe above 30%: a chunk's steps wait for one another.
#include <cuda_runtime.h>

#include <type_traits>

#include "sscan_heads.cuh"
#include "sscan_plan.h"
#include "sscan_vec.cuh"

namespace sscan {

__device__ unsigned int g_device_error_walk = 0;

namespace {

enum { kWalkOut = 0, kWalkLocal = 1, kWalkLocalRev = 2 };

template <typename T, int NT, int MODE>
struct Walk {
    static constexpr bool out = MODE == kWalkOut, bf16 = !Mma<T>::kExact32;
    // 128 states: two warps share 16 rows, each with half of the columns, which halves the
    // accumulators a warp holds
    static constexpr int WC = NT == 128 ? 2 : 1;
    static constexpr int NW = 4 * WC, threads = 32 * (NW + 1);
    // blocks per SM that shared memory allows, and registers are held to
    static constexpr int blocks = NT <= 32 ? 3 : NT == 64 ? (bf16 ? 3 : 2) : bf16 ? 2 : 1;
    static constexpr int stages = bf16 ? 2 : 1;  // buffers of tiles
    // From 64 states on, the state goes into the outputs as one bf16 part (its rounding is then the
    // same size as that of M on the other terms), the gate waits in registers, and the outputs
    // are staged in the rows of C that their own warps alone read: more blocks fit an SM.
    static constexpr bool big = bf16 && NT >= 64;
    // up to 32 states B is the smaller factor to scale, once per block through shared memory;
    // above, each warp scales its own 16 channels of u in registers
    static constexpr bool scale_b = bf16 && out && NT <= 32;
    static constexpr int PITCH_P = kHeadDim + Mma<T>::PAD, PITCH_N = NT + Mma<T>::PAD;

    struct Tiles {
        alignas(16) T x[kQ * PITCH_P];                       // u (reverse: dout)
        alignas(16) T B[kQ * PITCH_N];                       // B (reverse: C)
        alignas(16) T C[out ? kQ * PITCH_N : 8];
        alignas(16) T zr[MODE == kWalkLocalRev ? kQ * PITCH_P : 8];
    };
    struct Smem {
        Tiles t[stages];
        alignas(16) T z[out ? kQ * PITCH_P : 8];             // the gate, then the outputs
        alignas(16) T sh[out ? kHeadDim * PITCH_N : 8];      // the state, [p][n]
        alignas(16) T sl[out && bf16 && !big ? kHeadDim * PITCH_N : 8];
        alignas(16) T fb[scale_b ? 3 : 1][scale_b ? kQ * NT : 8];  // f B in three parts
        ChunkScalars s[2];
        unsigned int place;
    };
};

// A state handed from one segment's block to the next.
__device__ __forceinline__ bool wait_handed(const unsigned int* p, uint32_t limit = kWaitLimit) {
    for (uint32_t i = 0; i < limit; ++i) {
        unsigned int v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
        if (v) return true;
        __nanosleep(64);
    }
    return false;
}
__device__ __forceinline__ void hand_on(unsigned int* p) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(1u) : "memory");
}
__device__ __forceinline__ void raise_heads_error() { atomicOr(&g_device_error_walk, 1u); }

// barrier of the warps that run products (the scalars' warp stays out of it)
template <int THREADS>
__device__ __forceinline__ void product_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// The terms M_ts u_s, s <= t, of channel p whose u_s is not finite.
template <typename T>
__device__ __noinline__ float not_finite_terms(const T* C, const T* B, const T* x, const ChunkScalars& sc, int pn,
                                               int pp, int N, int t, int p) {
    float v = 0.f;
    for (int s = 0; s <= t; ++s) {
        const float xs = to_f32<T>(x[s * pp + p]);
        if (fabsf(xs) <= 3.4e38f) continue;
        float dot = 0.f;
        for (int m = 0; m < N; ++m) dot = fmaf(to_f32<T>(C[t * pn + m]), to_f32<T>(B[s * pn + m]), dot);
        v += dot * (chunk_decay(sc, t, s) * sc.w[s]) * xs;
    }
    return v;
}

// y = exp(c) C S^T + M U for 16 steps from t0 and 8 PTL channels from p0 of a chunk, the 16 columns
// s of M at a time, up to the diagonal.  FINITE: elements of U that are not finite count as 0.
template <typename T, int NT, int PTL, bool FINITE>
__device__ __forceinline__ void chunk_outputs(float (&y)[PTL][4], const T* C, const T* B, const T* x, const T* sh,
                                              const T* sl, const ChunkScalars& sc, int t0, int p0) {
    using M = Mma<T>;
    constexpr int PP = kHeadDim + M::PAD, PN = NT + M::PAD;
    const int g = (threadIdx.x & 31) >> 2, q = threadIdx.x & 3, ta = t0 + g, tb = ta + 8;
    zero_acc(y);
    warp_gemm<T, false, false, PTL>(y, C, PN, t0, sh, PN, p0, 0, NT);
    if constexpr (!M::kExact32 && NT < 64) warp_gemm<T, false, false, PTL>(y, C, PN, t0, sl, PN, p0, 0, NT);
    const float ea = sc.e[ta], eb = sc.e[tb];
#pragma unroll
    for (int j = 0; j < PTL; ++j) {
        y[j][0] *= ea, y[j][1] *= ea;
        y[j][2] *= eb, y[j][3] *= eb;
    }
    const float cha = sc.ch[ta], cla = sc.cl[ta], chb = sc.ch[tb], clb = sc.cl[tb];
    typename M::Addr x_at = M::at_bt(x, PP, p0);
#pragma unroll 1
    for (int s0 = 0; s0 <= t0; s0 += 16, x_at += M::template step_k<true>(PP) * (16 / M::KS)) {
        float m[2][4];
        zero_acc(m);
        warp_gemm<T, false, false, 2>(m, C, PN, t0, B, PN, s0, 0, NT);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int s = s0 + 8 * j + 2 * q;
            const float2 chs = *reinterpret_cast<const float2*>(sc.ch + s);
            const float2 cls = *reinterpret_cast<const float2*>(sc.cl + s);
            const float2 ws = *reinterpret_cast<const float2*>(sc.w + s);
            m[j][0] = s <= ta ? m[j][0] * (ex2((cha - chs.x) + (cla - cls.x)) * ws.x) : 0.f;
            m[j][1] = s + 1 <= ta ? m[j][1] * (ex2((cha - chs.y) + (cla - cls.y)) * ws.y) : 0.f;
            m[j][2] = s <= tb ? m[j][2] * (ex2((chb - chs.x) + (clb - cls.x)) * ws.x) : 0.f;
            m[j][3] = s + 1 <= tb ? m[j][3] * (ex2((chb - chs.y) + (clb - cls.y)) * ws.y) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 2; k += M::KT) {
            typename M::A fa;
            M::from_acc(fa, m + k);
#pragma unroll
            for (int j = 0; j < PTL; j += 2) {
                typename M::B b0, b1;
                M::template fetch_b2<true>(b0, b1, x_at + M::template step_k<true>(PP) * (k / M::KT) + M::template step_n<true>(PP) * (j / 2), PP);
                if constexpr (FINITE) M::keep_finite(b0), M::keep_finite(b1);
                M::mma(y[j], fa, b0);
                M::mma(y[j + 1], fa, b1);
            }
        }
    }
}

template <typename T, int NT, int MODE>
__global__ void __launch_bounds__(Walk<T, NT, MODE>::threads, Walk<T, NT, MODE>::blocks) heads_walk_kernel(const __grid_constant__ HeadsArgs a, const T* dout) {
    using W = Walk<T, NT, MODE>;
    using M = Mma<T>;
    constexpr int PP = W::PITCH_P, PN = W::PITCH_N, WC = W::WC, kWork = 32 * W::NW;
    constexpr int NTL = NT / 8 / WC, PTL = kHeadDim / 8 / WC;   // accumulator tiles of a warp
    constexpr bool kRev = MODE == kWalkLocalRev;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<typename W::Smem*>(smem_raw);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int wr = w / WC, wc = w % WC;
    // Blocks of a split sequence run in any order; where segments hand their state on, a ticket gives
    // them their place, segments in time order, so that the one a block waits for has started.
    int64_t b = blockIdx.y, seg = blockIdx.x / a.H;
    int h = (int)(blockIdx.x - seg * a.H);
    if (MODE == kWalkOut && a.ticket) {
        if (tid == 0) sm.place = atomicAdd(a.ticket, 1u);
        __syncthreads();
        const unsigned int all = (unsigned int)(a.batch * a.H), s = sm.place / all, r = sm.place - s * all;
        seg = s, b = r / a.H, h = (int)(r - b * a.H);
    }
    const int grp = h / (a.H / a.G);
    const int64_t c0 = seg * a.seg_chunks, c1 = c0 + a.seg_chunks < a.chunks ? c0 + a.seg_chunks : a.chunks;
    const int64_t bh = b * a.H + h, n = c1 - c0;
    const T *u = static_cast<const T*>(kRev ? (const void*)dout : a.u), *z = static_cast<const T*>(a.z);
    const T *Bm = static_cast<const T*>(kRev ? a.C : a.B), *Cm = static_cast<const T*>(a.C);
    auto chunk = [&](int64_t i) { return kRev ? c1 - 1 - i : c0 + i; };

    if (w == W::NW) {
        // the scalars of chunk i + 1 while the others work on chunk i
        chunk_scalars<T>(sm.s[0], a, b, h, chunk(0) * kQ);
        for (int64_t i = 0; i < n; ++i) {
            __syncthreads();
            if (i + 1 < n) chunk_scalars<T>(sm.s[(i + 1) & 1], a, b, h, chunk(i + 1) * kQ);
            if (W::stages == 1) __syncthreads();
        }
        return;
    }

    auto fetch = [&](int64_t i) {
        const int64_t t0 = chunk(i) * kQ, rows = a.L - t0 < kQ ? a.L - t0 : kQ;
        const int64_t row = (b * a.L + t0) * a.H + h, rowg = (b * a.L + t0) * a.G + grp;
        auto& t = sm.t[W::stages == 2 ? i & 1 : 0];
        load_tile_async<T, kHeadDim>(t.x, PP, u + row * a.P, (int64_t)a.H * a.P, rows, a.P, a.vec, tid, kWork);
        load_tile_async<T, NT>(t.B, PN, Bm + rowg * a.N, (int64_t)a.G * a.N, rows, a.N, a.vec, tid, kWork);
        if (W::out) load_tile_async<T, NT>(t.C, PN, Cm + rowg * a.N, (int64_t)a.G * a.N, rows, a.N, a.vec, tid, kWork);
        if (kRev && z)
            load_tile_async<T, kHeadDim>(t.zr, PP, z + row * a.P, (int64_t)a.H * a.P, rows, a.P, a.vec, tid, kWork);
    };

    // the state: rows p = 16 wr + g and + 8, columns n = (NT / WC) wc + 8 j + 2 q and + 1
    const int p0 = 16 * wr, n0 = NT / WC * wc;
    float S[NTL][4];
    zero_acc(S);
    auto each_state = [&](auto&& fn) {
#pragma unroll
        for (int j = 0; j < NTL; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = p0 + g + (i >> 1) * 8, m = n0 + 8 * j + 2 * q + (i & 1);
                if (p < a.P && m < a.N) fn(S[j][i], (int64_t)p * a.N + m);
            }
    };
    const bool handed = MODE == kWalkOut && a.ticket && seg > 0;
    auto entering = [&]() -> const float* {  // null: zero
        return MODE != kWalkOut          ? nullptr
               : handed                  ? a.states + (bh * a.nseg + seg - 1) * a.P * a.N
               : a.nseg > 1 && !a.ticket ? a.states + (bh * a.nseg + seg) * a.P * a.N
               : a.h0                    ? a.h0 + bh * a.P * a.N
                                         : nullptr;
    };
    if (MODE == kWalkOut) {
        const float* first = entering();
        if (W::stages == 2) {
            fetch(0);
            cp_async_commit();
        }
        if (handed) {
            if (tid == 0 && in_range(bh * a.nseg + seg - 1, segments(a)) && !wait_handed(a.handed + bh * a.nseg + seg - 1)) raise_heads_error();
            product_sync<kWork>();
        }
        if (first) {
            const int64_t base = handed ? bh * a.nseg + seg - 1 : a.nseg > 1 && !a.ticket ? bh * a.nseg + seg : bh;
            const int64_t extent = a.nseg > 1 && (handed || !a.ticket) ? states_extent(a) : state_extent(a);
            each_state([&](float& v, int64_t at) {
                if (in_range(base * a.P * a.N + at, extent)) v = __ldcg(first + at);
            });
        }
    }
    double total = 0.0;
    if (MODE != kWalkOut && W::stages == 2) {
        fetch(0);
        cp_async_commit();
    }

    for (int64_t i = 0; i < n; ++i) {
        const int64_t t0 = chunk(i) * kQ, rows = a.L - t0 < kQ ? a.L - t0 : kQ;
        const int64_t row = (b * a.L + t0) * a.H + h;
        auto& t = sm.t[W::stages == 2 ? i & 1 : 0];
        if (W::stages == 1) {
            __syncthreads();  // the last chunk's readers are done
            fetch(i);
            cp_async_commit();
        }
        cp_async_wait<0>();
        __syncthreads();      // this chunk's tiles and scalars are here; with two buffers, the other one is free
        const ChunkScalars& sc = sm.s[i & 1];
        if constexpr (W::out) {
            // the gate: a warp's own 16 steps (and, with two warps on them, both halves)
            if (z && !W::big)
                load_rows_async<T>(sm.z + p0 * PP, PP, z + (row + (int64_t)p0 * a.H) * a.P, (int64_t)a.H * a.P, rows - p0,
                                   a.P, a.vec);
            cp_async_commit();
        }
        if (W::stages == 2) {
            if (i + 1 < n) fetch(i + 1);
            cp_async_commit();
        }

        if constexpr (W::out) {
            // the state as the outputs read it, and f B
#pragma unroll
            for (int j = 0; j < NTL; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int at = (p0 + g + 8 * k) * PN + n0 + 8 * j + 2 * q;
                    const float x = S[j][2 * k], y = S[j][2 * k + 1];
                    if constexpr (W::big) *reinterpret_cast<uint32_t*>(sm.sh + at) = M::pack(x, y);
                    else split_store2<T>(sm.sh, sm.sl, at, x, y);
                }
            if constexpr (W::scale_b) {
#pragma unroll
                for (int k = tid; k < kQ * NT / 2; k += kWork) {
                    const int s = k / (NT / 2), n = (k - s * (NT / 2)) * 2, at = s * NT + n;
                    const uint32_t v = *reinterpret_cast<const uint32_t*>(t.B + s * PN + n);
                    float x = __uint_as_float(v << 16) * sc.f[s], y = __uint_as_float(v & 0xffff0000u) * sc.f[s];
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
                        const uint32_t r = Mma<__nv_bfloat16>::pack(x, y);
                        *reinterpret_cast<uint32_t*>(sm.fb[part] + at) = r;
                        x -= __uint_as_float(r << 16);
                        y -= __uint_as_float(r & 0xffff0000u);
                    }
                }
            }
            product_sync<kWork>();

            float y[PTL][4];
            const int c_p = kHeadDim / WC * wc;
            const int ta = p0 + g, tb = ta + 8;              // the rows of y are steps
            Vec<T, 2> zr[W::big ? PTL : 1][2];
            if (W::big && z) {
#pragma unroll
                for (int j = 0; j < PTL; ++j)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int st = k ? tb : ta, p = c_p + 8 * j + 2 * q;
                        const int64_t at = (row + (int64_t)st * a.H) * a.P + p;
                        zr[j][k].zero();
                        if (st < rows && p < a.P) {
                            if (a.vec) {
                                zr[j][k].load(z + at);
                            } else {
                                const float two[2] = {IO<T>::load(z, at), p + 1 < a.P ? IO<T>::load(z, at + 1) : 0.f};
                                zr[j][k].set(two);
                            }
                        }
                    }
            }
            const T* sl = W::bf16 ? sm.sl : nullptr;
            chunk_outputs<T, NT, PTL, false>(y, t.C, t.B, t.x, sm.sh, sl, sc, p0, c_p);
            // A value of u that is not finite meets the zeros of M above the diagonal in the product.
            // Where a result is not finite, the product is taken again without such values and the
            // terms that do hold them are added: they reach no earlier step.
            float probe = 0.f;
#pragma unroll
            for (int j = 0; j < PTL; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) probe = fmaf(y[j][k], 0.f, probe);
            if (__any_sync(0xffffffffu, probe != 0.f)) {
                chunk_outputs<T, NT, PTL, true>(y, t.C, t.B, t.x, sm.sh, sl, sc, p0, c_p);
#pragma unroll
                for (int j = 0; j < PTL; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        y[j][k] += not_finite_terms(t.C, t.B, t.x, sc, PN, PP, a.N, k < 2 ? ta : tb,
                                                    c_p + 8 * j + 2 * q + (k & 1));
            }
            // skip term and gate, through rows of shared memory to 16-byte stores
            if (!W::big) {
                if (W::stages == 2) cp_async_wait<1>();
                else cp_async_wait<0>();
            }
            if (WC > 1) product_sync<kWork>();
            else __syncwarp();
            T* stage = W::big ? t.C : sm.z;
            constexpr int PS = W::big ? PN : PP;
            const float D = head_param(a, a.D, h);
#pragma unroll
            for (int j = 0; j < PTL; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int st = k ? tb : ta, p = c_p + 8 * j + 2 * q;
                    float xv[2], v[2] = {y[j][2 * k], y[j][2 * k + 1]};
                    load_shared<2>(t.x + st * PP + p, xv);
                    if (a.D) v[0] = fmaf(D, xv[0], v[0]), v[1] = fmaf(D, xv[1], v[1]);
                    if (z) {
                        float zv[2];
                        if constexpr (W::big) zr[j][k].get(zv);
                        else load_shared<2>(sm.z + st * PP + p, zv);
                        v[0] *= silu(zv[0]), v[1] *= silu(zv[1]);
                    }
                    store_vec<2>(stage + st * PS + p, v);
                }
            __syncwarp();
            constexpr int VE = 16 / sizeof(T), PER = kHeadDim / WC / VE;
            T* out = static_cast<T*>(a.out);
#pragma unroll
            for (int k = lane; k < 16 * PER; k += 32) {
                const int r = k / PER, st = p0 + r, p = c_p + (k - r * PER) * VE;
                if (st >= rows || p >= a.P) continue;
                const int64_t at = (row + (int64_t)st * a.H) * a.P + p;
                if (a.vec) {
                    *reinterpret_cast<uint4*>(out + at) = *reinterpret_cast<const uint4*>(stage + st * PS + p);
                } else {
#pragma unroll
                    for (int v = 0; v < VE; ++v)
                        if (p + v < a.P) out[at + v] = stage[st * PS + p + v];
                }
            }
        }

        // S' = exp(c_end) S + (f U)^T B
        const float dec = ex2(sc.total * kLog2e);
        total += sc.total;
        float acc[NTL][4];
        zero_acc(acc);
        if constexpr (W::scale_b) {
#pragma unroll
            for (int k = 0; k < kQ; k += M::KS) {
                typename M::A fa;
                M::template fetch_a<true>(fa, M::at_at(t.x, PP, p0) + M::template step_k<true>(PP) * (k / M::KS), PP);
#pragma unroll
                for (int part = 2; part >= 0; --part)
#pragma unroll
                    for (int j = 0; j < NTL; j += 2) {
                        typename M::B b0, b1;
                        M::template fetch_b2<true>(b0, b1, M::at_bt(sm.fb[part], NT, n0) + M::template step_k<true>(NT) * (k / M::KS) + M::template step_n<true>(NT) * (j / 2), NT);
                        M::mma(acc[j], fa, b0);
                        M::mma(acc[j + 1], fa, b1);
                    }
            }
        } else {
            float lo[W::bf16 ? 1 : NTL][4];
            zero_acc(lo);
            typename M::Addr b_at = M::at_bt(t.B, PN, n0);
#pragma unroll 1
            for (int k = 0; k < kQ; k += M::KS, b_at += M::template step_k<true>(PN)) {
                Split<T> fa;
                load_at_split(fa, t.x, PP, p0, k, [&](float v, int p, int s) {
                    if (!kRev) return v * sc.f[s];
                    return (z ? v * silu(to_f32<T>(t.zr[s * PP + p])) : v) * sc.e[s];
                });
#pragma unroll
                for (int j = 0; j < NTL; j += 2) {
                    typename M::B b0, b1;
                    M::template fetch_b2<true>(b0, b1, b_at + M::template step_n<true>(PN) * (j / 2), PN);
                    if constexpr (W::bf16) {
                        mma_split(acc[j], fa, b0);
                        mma_split(acc[j + 1], fa, b1);
                    } else {
                        mma_split(acc[j], lo[j], fa, b0);
                        mma_split(acc[j + 1], lo[j + 1], fa, b1);
                    }
                }
            }
            if constexpr (!W::bf16) {
#pragma unroll
                for (int j = 0; j < NTL; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[j][k] += lo[j][k];
            }
        }
#pragma unroll
        for (int j = 0; j < NTL; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) S[j][k] = fmaf(dec, S[j][k], acc[j][k]);
    }
    // an infinity or a NaN stays in the state once it is there
    bool lost = false;
#pragma unroll
    for (int j = 0; j < NTL; ++j) lost = lost || not_finite(S[j]);
    auto mend = [&](float* dest) {
        if (kRev || !lost) return;
        auto place = [p = p0 + g, m = n0 + 2 * q](int j) { return make_int2(p + (j >> 1 & 1) * 8, m + 8 * (j >> 2) + (j & 1)); };
        const int64_t end = c1 * kQ;
        state_by_steps<T, 4 * NTL>(dest, place, a, b, h, c0 * kQ, end < a.L ? end : a.L, entering());
    };
    if (MODE == kWalkOut) {
        if (a.h_last && seg == a.nseg - 1) {
            float* o = a.h_last + bh * a.P * a.N;
            each_state([&](float& v, int64_t at) {
                if (in_range(bh * a.P * a.N + at, state_extent(a))) o[at] = v;
            });
            mend(o);
        }
        if (a.ticket && seg < a.nseg - 1) {
            float* o = a.states + (bh * a.nseg + seg) * a.P * a.N;
            each_state([&](float& v, int64_t at) {
                if (in_range((bh * a.nseg + seg) * a.P * a.N + at, states_extent(a))) __stcg(o + at, v);
            });
            mend(o);
            __syncwarp();
            __threadfence();
            product_sync<kWork>();
            if (tid == 0 && in_range(bh * a.nseg + seg, segments(a))) hand_on(a.handed + bh * a.nseg + seg);
        }
    } else {
        float* o = a.states + (bh * a.nseg + seg) * a.P * a.N;
        each_state([&](float& v, int64_t at) {
            if (in_range((bh * a.nseg + seg) * a.P * a.N + at, states_extent(a))) o[at] = v;
        });
        mend(o);
        if (tid == 0 && in_range(bh * a.nseg + seg, segments(a))) a.decays[bh * a.nseg + seg] = (float)total;
    }
}

// 8 x 24 pairs, 32 chunks, 64 x 64 states: 30 us for 201 MB, each state read and written once.
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
    for (int v = 0; v < V; ++v) cur[v] = first && in_range(bh * PN + at + v, state_extent(a)) ? first[bh * PN + at + v] : 0.f;
    auto held = [&](int64_t s) { return in_range((bh * a.nseg + s) * PN + at, states_extent(a), V); };
    constexpr int kAhead = 8;
    for (int64_t k0 = 0; k0 < a.nseg; k0 += kAhead) {
        Vec<float, V> loc[kAhead];
        float d[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (k0 + k < a.nseg) {
                const int64_t s = reverse ? a.nseg - 1 - (k0 + k) : k0 + k;
                loc[k].zero();
                if (held(s)) loc[k].load_rw(st + s * PN);
                d[k] = in_range(bh * a.nseg + s, segments(a)) ? dec[s] : 0.f;
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (k0 + k < a.nseg) {
                const int64_t s = reverse ? a.nseg - 1 - (k0 + k) : k0 + k;
                float x[V];
                loc[k].get(x);
                if (held(s)) store_vec<V>(st + s * PN, cur);
                const float e = ex2(d[k] * kLog2e);
#pragma unroll
                for (int v = 0; v < V; ++v)  // (an infinity is not decayed: e may have underflowed)
                    cur[v] = fmaf(fabsf(cur[v]) > 3.4e38f ? 1.f : e, cur[v], x[v]);
            }
    }
    if (last) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (in_range(bh * PN + at + v, state_extent(a))) last[bh * PN + at + v] = cur[v];
    }
}

// One token.  It moves 8 N bytes of state per channel and is bound by HBM bandwidth.  LPR lanes
// share the N states of a channel, four neighbouring ones each (V = 4, one 16-byte access) or one
// at a time; a warp takes kStepRows channels per lane group of one (batch, head), so that the
// scalars of that pair, some 80 instructions, are worked out once for 4 kStepRows states.  64 sequences,
// 80 heads of 64 channels, 16 states: 11 us for 44 MB (4.0 TB/s, in part from L2).
constexpr int kStepRows = 4;

template <typename T, int LPR, int V>
__global__ void __launch_bounds__(128) heads_step_kernel(HeadsArgs a, float* state, int units) {
    constexpr int RW = 32 / LPR;  // channels side by side in a warp
    const int lane = threadIdx.x & 31, r0 = lane / LPR, l = lane % LPR;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t bh = unit / units;
    if (bh >= a.batch * a.H) return;
    const int p0 = (int)(unit - bh * units) * RW * kStepRows + r0;
    const int64_t b = bh / a.H;
    const int h = (int)(bh - b * a.H);
    const int64_t bg = b * a.G + h / (a.H / a.G);
    const T *Bp = static_cast<const T*>(a.B) + bg * a.N, *Cp = static_cast<const T*>(a.C) + bg * a.N;

    float x[kStepRows], zv[kStepRows];
    Vec<float, V> s[kStepRows];
    auto held = [&](int p, int n) { return in_range((bh * a.P + p) * a.N + n, state_extent(a), V); };
    const bool one = V * LPR >= a.N;  // every state of a channel is in one access of its lanes
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) {
        const int p = p0 + k * RW;
        if (p >= a.P) continue;
        s[k].zero();
        if (one && l * V < a.N && held(p, l * V)) s[k].load_rw(state + (bh * a.P + p) * a.N + l * V);
        x[k] = IO<T>::load(static_cast<const T*>(a.u), bh * a.P + p);
        zv[k] = a.z ? IO<T>::load(static_cast<const T*>(a.z), bh * a.P + p) : 0.f;
    }
    const float A = head_param(a, a.A, h), D = head_param(a, a.D, h);
    const float r = IO<T>::load(static_cast<const T*>(a.delta_raw), bh) + head_param(a, a.bias, h);
    const float dl = a.softplus ? (r > 20.f ? r : log1pf(expf(r))) : r;
    const float qv = dl * A, dec = ex2(qv * kLog2e), w = A != 0.f ? expm1f(qv) / A : dl;
    float y[kStepRows];
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) y[k] = 0.f;
    for (int n = l * V; n < a.N; n += LPR * V) {
        float Bn[V], Cn[V];
#pragma unroll
        for (int v = 0; v < V; ++v) Bn[v] = IO<T>::load(Bp, n + v), Cn[v] = IO<T>::load(Cp, n + v);
#pragma unroll
        for (int k = 0; k < kStepRows; ++k) {
            const int p = p0 + k * RW;
            if (p >= a.P) continue;
            float* sp = state + (bh * a.P + p) * a.N + n;
            if (!one && held(p, n)) s[k].load_rw(sp);
            float sv[V];
            s[k].get(sv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                sv[v] = fmaf(dec, sv[v], w * x[k] * Bn[v]);
                y[k] = fmaf(sv[v], Cn[v], y[k]);
            }
            if (held(p, n)) store_vec<V>(sp, sv);
        }
    }
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) {
#pragma unroll
        for (int o = 1; o < LPR; o *= 2) y[k] += __shfl_xor_sync(0xffffffffu, y[k], o);
        const int p = p0 + k * RW;
        if (l == 0 && p < a.P) {
            float v = a.D ? fmaf(D, x[k], y[k]) : y[k];
            if (a.z) v *= silu(zv[k]);
            IO<T>::store(static_cast<T*>(a.out), bh * a.P + p, v);
        }
    }
}

// wait_handed made to run out of polls, on a flag that nothing sets.
__device__ unsigned int g_probe_flag = 0;
__global__ void handed_probe_kernel(unsigned int polls) {
    if (!wait_handed(&g_probe_flag, polls)) atomicOr(&g_device_error_walk, 4u);
}

// ---------------------------------------------------------------- host

template <typename T, int NT, int MODE>
cudaError_t walk(const HeadsArgs& a, const void* dout, cudaStream_t st) {
    auto* k = heads_walk_kernel<T, NT, MODE>;
    using W = Walk<T, NT, MODE>;
    constexpr size_t smem = sizeof(typename W::Smem);
    static_assert(smem <= 227 * 1024, "the tiles of one chunk must fit a block's shared memory");
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    k<<<dim3((unsigned)(a.H * a.nseg), (unsigned)a.batch), W::threads, smem, st>>>(a, static_cast<const T*>(dout));
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

template <typename T, int LPR, int V>
void step_heads(const HeadsArgs& a, float* state, cudaStream_t st) {
    constexpr int per = 32 / LPR * kStepRows;
    const int units = (a.P + per - 1) / per;
    heads_step_kernel<T, LPR, V><<<(unsigned)((a.batch * a.H * units + 3) / 4), 128, 0, st>>>(a, state, units);
}

// Four states per lane where rows of the state are 16-byte aligned, with as many lanes per
// channel as that takes (a power of two).
template <typename T>
void launch_step_heads(const HeadsArgs& a, float* state, cudaStream_t st) {
    if (a.N % 4 == 0 && aligned_to(state, 16)) {
        if (a.N <= 16) step_heads<T, 4, 4>(a, state, st);
        else if (a.N <= 32) step_heads<T, 8, 4>(a, state, st);
        else if (a.N <= 64) step_heads<T, 16, 4>(a, state, st);
        else step_heads<T, 32, 4>(a, state, st);
    } else if (a.N <= 8) {
        step_heads<T, 8, 1>(a, state, st);
    } else {
        step_heads<T, 32, 1>(a, state, st);
    }
}

// Blocks of the output kernel that the GPU holds at once.
int64_t heads_slots(const HeadsArgs& a, bool bf16) {
    auto per = [&](auto t) {
        using T = decltype(t);
        return a.N <= 16 ? Walk<T, 16, kWalkOut>::blocks : a.N <= 32 ? Walk<T, 32, kWalkOut>::blocks
               : a.N <= 64 ? Walk<T, 64, kWalkOut>::blocks : Walk<T, 128, kWalkOut>::blocks;
    };
    return kSmCount * (int64_t)(bf16 ? per(__nv_bfloat16{}) : per(float{}));
}

// Segments of a forward pass.  With fewer (batch, head) pairs than SMs a sequence is split into as
// many segments, of at least four chunks, as fill the GPU once: a block more than it holds would
// wait for a whole segment (65536 steps, 24 heads: with 32 states, where 444 blocks fit, 18 segments,
// 432 blocks, 530 us, 27 segments 682 us; with 128 states on tcgen05, where 148 fit, 6 segments 621 us,
// 9 segments 819 us).  From one pair per SM on it is not split, which leaves slots empty up to where segments are
// handed on: 16 states, 16384 steps, 147 / 148 / 160 / 220 pairs take 587 / 859 / 1000 / 1019 us, and with a split up to
// half the slots 587 / 586 / 849 / 876 us.
void plan_segments(HeadsArgs& a, int64_t slots, int64_t least) {
    const int64_t bh = a.batch * a.H;
    int64_t nseg = 1;
    if (bh < kSmCount) {
        nseg = slots / bh;
        if (nseg > (a.chunks + least - 1) / least) nseg = (a.chunks + least - 1) / least;
        if (nseg < 2) nseg = 1;
    }
    a.seg_chunks = (a.chunks + nseg - 1) / nseg;
    a.nseg = (a.chunks + a.seg_chunks - 1) / a.seg_chunks;
}

// Whether the tcgen05 kernel takes this problem, pointers (a.vec) aside, and its plan: one block per SM.
bool tc_problem(const HeadsArgs& a, bool bf16) { return bf16 && a.N > 32 && a.L < (int64_t(1) << 31) - kTcQ; }

// More (batch, head) pairs than the GPU holds blocks: segments of 8 chunks hand their state on, so that
// the last wave is a few chunks long instead of a whole sequence (8 x 2048, 80 heads, 640 pairs where
// 444 blocks fit).  With fewer pairs a block would wait for the one before it.
constexpr int64_t kHandedChunks = 8;
bool hands_on(const HeadsArgs& a, bool bf16) {
    return a.batch * a.H > heads_slots(a, bf16) && a.chunks > kHandedChunks;
}

void plan_heads(HeadsArgs& a, bool bf16, bool tc) {
    if (tc) a.chunks = (a.L + kTcQ - 1) / kTcQ;
    if (!tc && hands_on(a, bf16)) {
        a.seg_chunks = kHandedChunks;
        a.nseg = (a.chunks + kHandedChunks - 1) / kHandedChunks;
        return;
    }
    plan_segments(a, tc ? kSmCount : heads_slots(a, bf16), tc ? 2 : 4);
}

size_t split_bytes(const HeadsArgs& a) {
    const size_t bh = (size_t)(a.batch * a.H);
    return round256(bh * a.nseg * a.P * a.N * sizeof(float)) + round256((bh * a.nseg + 1) * sizeof(float));
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

cudaError_t launch_handed_probe(unsigned int polls, cudaStream_t st) {
    handed_probe_kernel<<<1, 1, 0, st>>>(polls);
    return cudaGetLastError();
}

cudaError_t read_device_error_walk(unsigned int* value, int clear) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error_walk, sizeof(unsigned int));
    if (e == cudaSuccess && clear && *value) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_device_error_walk, &zero, sizeof(unsigned int));
    }
    return e;
}

size_t heads_fwd_bytes(const sscan_heads_problem* p) {
    HeadsArgs a = heads_args(p, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
    const bool bf16 = p->io_dtype == SSCAN_BF16;
    HeadsArgs t = a;  // either kernel may take the call, by its pointers
    plan_heads(a, bf16, false);
    size_t bytes = a.nseg > 1 ? split_bytes(a) : 0;
    if (tc_problem(t, bf16)) {
        plan_heads(t, bf16, true);
        if (t.nseg > 1 && split_bytes(t) > bytes) bytes = split_bytes(t);
    }
    return bytes;
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
    a.vec = a.vec && aligned_to(z, 16) && aligned_to(out, 16);
    const bool bf16 = p->io_dtype == SSCAN_BF16;
    const bool tc = a.vec && tc_problem(a, bf16);
    plan_heads(a, bf16, tc);
    cudaError_t e = cudaSuccess;
    if (a.nseg > 1) {
        a.states = static_cast<float*>(workspace);
        a.decays = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                            round256((size_t)(a.batch * a.H * a.nseg * a.P * a.N) * sizeof(float)));
    }
    if (a.nseg > 1 && !tc && hands_on(a, bf16)) {
        a.ticket = reinterpret_cast<unsigned int*>(a.decays);
        a.handed = a.ticket + 1;
        e = cudaMemsetAsync(a.ticket, 0, (size_t)(a.batch * a.H * a.nseg + 1) * sizeof(unsigned int), st);
        if (e != cudaSuccess) return api_fail(SSCAN_ERR_CUDA, "clearing the segments' flags: %s", cudaGetErrorString(e));
    } else if (a.nseg > 1) {
        e = tc ? launch_heads_tc(a, true, st) : launch_heads_local(a, nullptr, bf16, st);
        if (e != cudaSuccess) return api_fail(SSCAN_ERR_CUDA, "segment state kernel: %s", cudaGetErrorString(e));
        launch_heads_carry(a, false, h0, nullptr, st);
        if (sscan_status s = api_launched("segment carry kernel")) return s;
    }
    e = tc ? launch_heads_tc(a, false, st)
        : bf16 ? walk_n<__nv_bfloat16, kWalkOut>(a, nullptr, st) : walk_n<float, kWalkOut>(a, nullptr, st);
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
    if (p->io_dtype == SSCAN_BF16) launch_step_heads<__nv_bfloat16>(a, state, st);
    else launch_step_heads<float>(a, state, st);
    api_count_launch();
    return api_launched("heads step kernel");
}

}  // extern "C"
