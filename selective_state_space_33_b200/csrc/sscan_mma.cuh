// sscan_mma.cuh -- warp-level matrix products over shared-memory tiles for the multi-head
// recurrence: one interface over bf16 operands and over fp32 operands, accumulating in fp32.
//
// Element (row, k) of A and (k, col) of B come from row-major tiles, either as stored or
// transposed.  bf16: m16n8k16 instructions, fragments by ldmatrix.  fp32: m16n8k8 tf32
// instructions on operands split in two tf32 parts, x = hi + lo with |lo| <= 2^-11 |x|; the
// three products hi hi, hi lo, lo hi leave out lo lo, a relative 2^-22.  The k slots of an
// fp32 fragment are permuted (slot t holds k = 2t, slot t + 4 holds k = 2t + 1) so that an
// accumulator is an A fragment as it stands.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace sscan {

template <int NTL>
__device__ __forceinline__ void zero_acc(float (&acc)[NTL][4]) {
#pragma unroll
    for (int j = 0; j < NTL; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
}

template <typename T> struct Mma;

template <> struct Mma<__nv_bfloat16> {
    using T = __nv_bfloat16;
    static constexpr int KS = 16;   // k per instruction
    static constexpr int KT = 2;    // 8-wide accumulator tiles per A fragment
    static constexpr int PAD = 8;   // elements added to a tile's row pitch: 16 bytes, so that eight
                                    // consecutive rows start in eight different 16-byte bank groups
    static constexpr bool kExact32 = false;
    struct A { uint32_t r[4]; };
    struct B { uint32_t r[2]; };

    // Where a lane's ldmatrix row starts, for k = 0: the four ways an operand can be stored, as
    // shared-memory byte addresses, and how far k .. k + 15 and the next 16 columns are from there.
    using Addr = uint32_t;
    static __device__ __forceinline__ Addr addr(const T* p) {
        return static_cast<uint32_t>(__cvta_generic_to_shared(p));
    }
    static __device__ __forceinline__ Addr at_a(const T* s, int pitch, int m0) {   // [m][k]
        const int l = threadIdx.x & 31;
        return addr(s + (m0 + (l & 15)) * pitch + (l >> 4) * 8);
    }
    static __device__ __forceinline__ Addr at_at(const T* s, int pitch, int m0) {  // [k][m]
        const int l = threadIdx.x & 31;
        return addr(s + ((l & 7) + (l >> 4) * 8) * pitch + m0 + ((l >> 3) & 1) * 8);
    }
    static __device__ __forceinline__ Addr at_b(const T* s, int pitch, int n0) {   // [n][k]
        const int l = threadIdx.x & 31;
        return addr(s + (n0 + (l & 7) + (l >> 4) * 8) * pitch + ((l >> 3) & 1) * 8);
    }
    static __device__ __forceinline__ Addr at_bt(const T* s, int pitch, int n0) {  // [k][n]
        const int l = threadIdx.x & 31;
        return addr(s + (l & 15) * pitch + n0 + (l >> 4) * 8);
    }
    template <bool TR> static __device__ __forceinline__ Addr step_k(int pitch) { return TR ? 16 * pitch * 2 : 32; }
    template <bool TR> static __device__ __forceinline__ Addr step_n(int pitch) { return TR ? 32 : 16 * pitch * 2; }

    template <bool TR> static __device__ __forceinline__ void load4(uint32_t (&r)[4], Addr p) {
        if constexpr (TR)
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                         : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p) : "memory");
        else
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                         : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p) : "memory");
    }
    // 16 rows by 16 k
    template <bool TR> static __device__ __forceinline__ void fetch_a(A& a, Addr p, int) { load4<TR>(a.r, p); }
    // 16 k by 16 columns: two fragments
    template <bool TR> static __device__ __forceinline__ void fetch_b2(B& b0, B& b1, Addr p, int) {
        uint32_t r[4];
        load4<TR>(r, p);
        b0.r[0] = r[0], b0.r[1] = r[1], b1.r[0] = r[2], b1.r[1] = r[3];
    }
    // infinities and NaN (all exponent bits set) become 0
    static __device__ __forceinline__ void keep_finite(B& b) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if ((b.r[i] & 0x7f80u) == 0x7f80u) b.r[i] &= 0xffff0000u;
            if ((b.r[i] & 0x7f800000u) == 0x7f800000u) b.r[i] &= 0xffffu;
        }
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    // accumulator tiles c[0], c[1] (16 rows by 16 columns) as an A fragment, rounded to bf16
    static __device__ __forceinline__ void from_acc(A& a, const float (*c)[4]) {
        a.r[0] = pack(c[0][0], c[0][1]);
        a.r[1] = pack(c[0][2], c[0][3]);
        a.r[2] = pack(c[1][0], c[1][1]);
        a.r[3] = pack(c[1][2], c[1][3]);
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const A& a, const B& b) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a.r[0]), "r"(a.r[1]), "r"(a.r[2]), "r"(a.r[3]), "r"(b.r[0]), "r"(b.r[1]));
    }
};

template <> struct Mma<float> {
    using T = float;
    static constexpr int KS = 8;
    static constexpr int KT = 1;
    static constexpr int PAD = 4;
    static constexpr bool kExact32 = true;
    struct A { uint32_t hi[4], lo[4]; };
    struct B { uint32_t hi[2], lo[2]; };

    static __device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
        asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
        const float rest = x - __uint_as_float(hi);
        asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(rest));
    }
    static __device__ __forceinline__ void put(A& a, int i, float x) { split(x, a.hi[i], a.lo[i]); }
    // A lane's first element, for k = 0, as a pointer; the steps are in elements.
    using Addr = const float*;
    static __device__ __forceinline__ Addr at_a(const T* s, int pitch, int m0) {
        return s + (m0 + ((threadIdx.x & 31) >> 2)) * pitch + 2 * (threadIdx.x & 3);
    }
    static __device__ __forceinline__ Addr at_at(const T* s, int pitch, int m0) {
        return s + 2 * (threadIdx.x & 3) * pitch + m0 + ((threadIdx.x & 31) >> 2);
    }
    static __device__ __forceinline__ Addr at_b(const T* s, int pitch, int n0) { return at_a(s, pitch, n0); }
    static __device__ __forceinline__ Addr at_bt(const T* s, int pitch, int n0) { return at_at(s, pitch, n0); }
    template <bool TR> static __device__ __forceinline__ int step_k(int pitch) { return TR ? 8 * pitch : 8; }
    template <bool TR> static __device__ __forceinline__ int step_n(int pitch) { return TR ? 16 : 16 * pitch; }
    template <bool TR> static __device__ __forceinline__ void fetch_a(A& a, Addr p, int pitch) {
        const int m = TR ? 8 : 8 * pitch, k = TR ? pitch : 1;  // 8 rows on, one k on
        put(a, 0, p[0]);
        put(a, 1, p[m]);
        put(a, 2, p[k]);
        put(a, 3, p[m + k]);
    }
    template <bool TR> static __device__ __forceinline__ void fetch_b2(B& b0, B& b1, Addr p, int pitch) {
        const int n = TR ? 8 : 8 * pitch, k = TR ? pitch : 1;
        split(p[0], b0.hi[0], b0.lo[0]);
        split(p[k], b0.hi[1], b0.lo[1]);
        split(p[n], b1.hi[0], b1.lo[0]);
        split(p[n + k], b1.hi[1], b1.lo[1]);
    }
    static __device__ __forceinline__ void keep_finite(B& b) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if ((b.hi[i] & 0x7f800000u) == 0x7f800000u) b.hi[i] = b.lo[i] = 0u;
    }
    static __device__ __forceinline__ void from_acc(A& a, const float (*c)[4]) {
        put(a, 0, c[0][0]);
        put(a, 1, c[0][2]);
        put(a, 2, c[0][1]);
        put(a, 3, c[0][3]);
    }
    static __device__ __forceinline__ void one(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
        asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
    }
    static __device__ __forceinline__ void mma(float (&c)[4], float (&lo)[4], const A& a, const B& b) {
        one(lo, a.lo, b.hi);
        one(lo, a.hi, b.lo);
        one(c, a.hi, b.hi);
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const A& a, const B& b) {
        one(c, a.lo, b.hi);
        one(c, a.hi, b.lo);
        one(c, a.hi, b.hi);
    }
};

// acc[NTL][4] (16 rows m0.. by 8 NTL columns n0..) += A[m][k] B[k][n], k = k_begin .. k_end - 1.
// AT / BT: the operand's tile is stored [k][m] / [k][n] instead of [m][k] / [n][k].  NTL is even.
template <typename T, bool AT, bool BT, int NTL>
__device__ __forceinline__ void warp_gemm(float (&acc)[NTL][4], const T* A, int pa, int m0, const T* B, int pb, int n0,
                                          int k_begin, int k_end) {
    using M = Mma<T>;
    typename M::Addr a_at = AT ? M::at_at(A, pa, m0) : M::at_a(A, pa, m0);
    typename M::Addr b_at = BT ? M::at_bt(B, pb, n0) : M::at_b(B, pb, n0);
    a_at += M::template step_k<AT>(pa) * (k_begin / M::KS);
    b_at += M::template step_k<BT>(pb) * (k_begin / M::KS);
    // fp32: the corrections hi lo + lo hi gather apart from the products of the leading parts, which
    // the tensor core's accumulation then truncates a third as often
    float lo[M::kExact32 ? NTL : 1][4];
    if constexpr (M::kExact32) zero_acc(lo);
#pragma unroll 4
    for (int k = k_begin; k < k_end; k += M::KS) {
        typename M::A a;
        M::template fetch_a<AT>(a, a_at, pa);
#pragma unroll
        for (int j = 0; j < NTL; j += 2) {
            typename M::B b0, b1;
            M::template fetch_b2<BT>(b0, b1, b_at + M::template step_n<BT>(pb) * (j / 2), pb);
            if constexpr (M::kExact32) {
                M::mma(acc[j], lo[j], a, b0);
                M::mma(acc[j + 1], lo[j + 1], a, b1);
            } else {
                M::mma(acc[j], a, b0);
                M::mma(acc[j + 1], a, b1);
            }
        }
        a_at += M::template step_k<AT>(pa);
        b_at += M::template step_k<BT>(pb);
    }
    if constexpr (M::kExact32) {
#pragma unroll
        for (int j = 0; j < NTL; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] += lo[j][i];
    }
}

// An A fragment of products v_i that are not exact in the tile type, as parts whose sum is v to
// 2^-24: three bf16 fragments, or the one fp32 fragment (itself two tf32 parts).
template <typename T> struct Split;
template <> struct Split<__nv_bfloat16> {
    static constexpr int PARTS = 3;
    Mma<__nv_bfloat16>::A part[3];
    __device__ __forceinline__ void set(int i, float x, float y) {  // register i: k and k + 1 of one row
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const uint32_t v = Mma<__nv_bfloat16>::pack(x, y);
            part[p].r[i] = v;
            x -= __uint_as_float(v << 16);
            y -= __uint_as_float(v & 0xffff0000u);
        }
    }
};
template <> struct Split<float> {
    static constexpr int PARTS = 1;
    Mma<float>::A part[1];
};

// The fragment at rows m0, k0 of a tile stored [k][m], every element passed through
// fn(value, row m, k) and split.
template <typename Fn>
__device__ __forceinline__ void load_at_split(Split<__nv_bfloat16>& a, const __nv_bfloat16* s, int pitch, int m0, int k0,
                                              Fn fn) {
    Mma<__nv_bfloat16>::A raw;
    Mma<__nv_bfloat16>::fetch_a<true>(raw, Mma<__nv_bfloat16>::at_at(s + k0 * pitch, pitch, m0), pitch);
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + g + (i & 1) * 8, k = k0 + 2 * t + (i >> 1) * 8;
        a.set(i, fn(__uint_as_float(raw.r[i] << 16), m, k), fn(__uint_as_float(raw.r[i] & 0xffff0000u), m, k + 1));
    }
}
template <typename Fn>
__device__ __forceinline__ void load_at_split(Split<float>& a, const float* s, int pitch, int m0, int k0, Fn fn) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
    const float* p = s + (k0 + 2 * t) * pitch + m0 + g;
    Mma<float>::put(a.part[0], 0, fn(p[0], m0 + g, k0 + 2 * t));
    Mma<float>::put(a.part[0], 1, fn(p[8], m0 + g + 8, k0 + 2 * t));
    Mma<float>::put(a.part[0], 2, fn(p[pitch], m0 + g, k0 + 2 * t + 1));
    Mma<float>::put(a.part[0], 3, fn(p[pitch + 8], m0 + g + 8, k0 + 2 * t + 1));
}

// acc += a b with every part of a, the small ones first.
__device__ __forceinline__ void mma_split(float (&acc)[4], const Split<__nv_bfloat16>& a, const Mma<__nv_bfloat16>::B& b) {
#pragma unroll
    for (int p = 2; p >= 0; --p) Mma<__nv_bfloat16>::mma(acc, a.part[p], b);
}
// fp32: products with the leading parts go to `acc`, the corrections to `lo`.  The tensor core's
// accumulation drops low bits at each step, so the small terms are kept apart, the large ones take a
// third of the steps, and the caller adds the two in fp32.
__device__ __forceinline__ void mma_split(float (&acc)[4], float (&lo)[4], const Split<float>& a, const Mma<float>::B& b) {
    Mma<float>::one(lo, a.part[0].lo, b.hi);
    Mma<float>::one(lo, a.part[0].hi, b.lo);
    Mma<float>::one(acc, a.part[0].hi, b.hi);
}

// 16 bytes from global to shared memory, asynchronously; zeros when !in (src is then not read).
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool in) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    const int n = in ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace sscan
