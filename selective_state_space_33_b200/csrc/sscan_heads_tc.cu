// sscan_heads_tc.cu -- the forward of the multi-head recurrence (sscan_heads.cuh) on the 5th-generation
// tensor cores, for bf16 I/O and more than 32 states.
//
// With 128 states the chunk's products are 2 x 128 x (128 + 3 x 64 + 64 + 64) x 128 operations against 48 KB
// of traffic; as mma.sync they kept eight warps loading fragments (1470 us at 65536 steps, 24 heads, 128
// states, issue slots 45% busy, tensor pipe under 40%).  Here one thread issues them from
// shared memory and tensor memory, and the warps only do what is elementwise: 621 us, about
// 72% of it the output pass and 27% the pass over the segments' states.  What is left is the order of a chunk's
// steps with one block per SM (output pass: issue slots 39%, tensor pipe 19% busy); barriers that keep the
// working warps in step are faster than mbarriers that let them drift (815 against 764 us at
// that stage: drifting warps miss the instruction cache).
//
// A block walks the chunks (128 steps) of one (batch, head, segment).  Tiles are rows of 64 bf16 in the
// 128-byte swizzle, as TMA writes them: such a tile is a K-major operand when its rows are
// the operand's rows and an MN-major one when its rows are k, so no tile is transposed:
//   G  = C B^T         rows t, columns s   (C, B K-major)                 tensor memory, 128 columns
//   Ya = C S^T         rows t, columns p   (C K-major, S [n][p] MN-major)                  64
//   Yb = M U           rows t, columns p   (M bf16 in tensor memory, U [s][p] MN-major)    64
//   St = B^T (f U)     rows n, columns p   (B [s][n], f U [s][p], both MN-major)           64
// y = exp(c) Ya + Yb.  f U goes in as three bf16 parts (24 bits: the state is an fp32 result), S and M
// as one, each a rounding of the size of the output's own.  The state itself stays in fp32
// registers, row n and a quarter of the channels per thread.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "sscan_heads.cuh"
#include "sscan_vec.cuh"

namespace sscan {

__device__ unsigned int g_device_error_heads = 0;

namespace {

using bf16 = __nv_bfloat16;

constexpr int kWork = 512;               // 16 warps: 4 quarters of the rows by 4 of the columns
constexpr int kIssuer = kWork / 32;      // index of the issuing warp
constexpr int kIssue = kWork + 32;       // and the warp that issues products and copies
constexpr int kThreads = kIssue + 64;    // and one each for the scalars of even and odd chunks
constexpr int kTile = kTcQ * 64;         // elements of a tile of 128 rows
constexpr uint32_t kColG = 0, kColM = 128, kColYa = 192, kColYb = 256, kColSt = 320, kCols = 512;

struct TcSmem {
    alignas(1024) bf16 x[2][kTile];      // by chunk, as B
    alignas(1024) bf16 B[2][2][kTile];   // states 0..63 and 64..127
    alignas(1024) bf16 C[2][kTile];
    alignas(1024) bf16 z[kTile];         // the gate, then the outputs
    alignas(1024) bf16 f[3][kTile];      // f U in three parts
    alignas(1024) bf16 S[kTile];         // [n][p]
    ChunkScalarsOf<kTcQ> s[4];           // by chunk
    alignas(8) uint64_t scalars_ready[4], scalars_free[4];
    uint64_t full_x[2], full_b[2], full_c, full_z, done_g, done_ya, done_st, done_yb;  // copies and products
    uint32_t tmem;
};

// --- tcgen05 -------------------------------------------------------------------------------

// Shared-memory operand: 128-byte swizzle; lead: bytes between blocks of 64 along the operand's rows
// or columns (MN-major only); groups of eight tile rows are 1024 bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// bf16 x bf16 -> fp32, 128 rows by n columns; ta / tb: the operand is MN-major.
__host__ __device__ constexpr uint32_t instruction(int n, int ta, int tb) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)ta << 15) | ((uint32_t)tb << 16) | ((uint32_t)(n / 8) << 17) |
           ((128u / 16) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 or 16 columns of this warp's 32 rows.
__device__ __forceinline__ void tmem_load(float (&v)[32], uint32_t at) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_load(float (&v)[16], uint32_t at) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int t, int b, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(t), "r"(b), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, int x, int y, int t, int b, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(t), "r"(b), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The working warps and the issuing one keep step: three barriers a chunk.
__device__ __forceinline__ void work_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kIssue) : "memory"); }
__device__ __forceinline__ int work_or(int v) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(v), "n"(kIssue) : "memory");
    return r;
}

// Byte offset of 16-byte unit c of row r of a tile.
__device__ __forceinline__ uint32_t unit(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ void widen8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}

// The outputs of a thread's 16 channels at step t of a chunk with values of u that are not finite: such
// values were left out of Yb, and the terms M_ts u_s that hold one are added for s <= t alone, from
// global memory.  A function of its own: inlined it costs the usual path about 1% (8 x 2048, 24 heads, 64
// states, forward and backward: 885 against 875 us; 65536 steps, 128 states: 641 against 639).
__device__ __noinline__ void rare_outputs(const HeadsArgs& a, const ChunkScalarsOf<kTcQ>& s, uint32_t ya_at, uint32_t yb_at,
                                          unsigned char* zb, int b, int h, int64_t t0, int t, int p0) {
    const bf16 *u = static_cast<const bf16*>(a.u), *B = static_cast<const bf16*>(a.B), *C = static_cast<const bf16*>(a.C);
    const int grp = h / (a.H / a.G);
    const float e = s.e[t], D = head_param(a, a.D, h);
    float ya[16], yb[16];
    tmem_load(ya, ya_at);
    tmem_load(yb, yb_at);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int p = p0 + j;
        bf16* z = reinterpret_cast<bf16*>(zb + unit(t, p / 8)) + p % 8;
        float v = fmaf(e, ya[j], yb[j]), x = 0.f;
        if (t0 + t < a.L && p < a.P) {
            x = __bfloat162float(u[((b * a.L + t0 + t) * a.H + h) * a.P + p]);
            for (int q = 0; q <= t; ++q) {
                const float uq = __bfloat162float(u[((b * a.L + t0 + q) * a.H + h) * a.P + p]);
                if (fabsf(uq) <= 3.4e38f) continue;
                float dot = 0.f;
                for (int n = 0; n < a.N; ++n)
                    dot = fmaf(__bfloat162float(C[((b * a.L + t0 + t) * a.G + grp) * a.N + n]),
                               __bfloat162float(B[((b * a.L + t0 + q) * a.G + grp) * a.N + n]), dot);
                v += dot * (chunk_decay(s, t, q) * s.w[q]) * uq;
            }
        }
        if (a.D) v = fmaf(D, x, v);
        if (a.z) v *= silu(__bfloat162float(*z));
        *z = __float2bfloat16_rn(v);
    }
}

// The state that enters a segment (null: zero).
template <bool kOut>
__device__ __forceinline__ const float* entering_state(const HeadsArgs& a, int64_t bh, int64_t seg) {
    if (!kOut) return nullptr;
    return a.nseg > 1 ? a.states + (bh * a.nseg + seg) * a.P * a.N : a.h0 ? a.h0 + bh * a.P * a.N : nullptr;
}

// state_by_steps of a working thread's 16 elements over the block's segment; everything it needs is worked out
// anew, which costs the usual path no registers.
template <bool kOut>
__device__ __noinline__ void segment_by_steps(const HeadsArgs& a) {
    const int64_t seg = blockIdx.x / a.H, b = blockIdx.y;
    const int h = (int)(blockIdx.x - seg * a.H), w = threadIdx.x >> 5;
    const int row = 32 * (w & 3) + (threadIdx.x & 31), p0 = 16 * (w >> 2);
    const int64_t t0 = seg * a.seg_chunks * kTcQ, end = t0 + a.seg_chunks * kTcQ, bh = b * a.H + h;
    float* dest = kOut ? a.h_last + bh * a.P * a.N : a.states + (bh * a.nseg + seg) * a.P * a.N;
    state_by_steps<bf16, 16>(dest, [p0, row](int k) { return make_int2(p0 + k, row); }, a, b, h, t0, end < a.L ? end : a.L,
                             entering_state<kOut>(a, bh, seg));
}

// kOut: outputs, from the state entering the segment; else the segment's end state from zero.
template <int NT, bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
    heads_tc_kernel(const __grid_constant__ CUtensorMap tm_u, const __grid_constant__ CUtensorMap tm_z,
                    const __grid_constant__ CUtensorMap tm_B, const __grid_constant__ CUtensorMap tm_C,
                    const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ HeadsArgs a) {
    constexpr int HALVES = NT / 64;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    auto& sm = *reinterpret_cast<TcSmem*>(smem_raw);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int64_t seg = blockIdx.x / a.H;
    const int b = blockIdx.y, h = (int)(blockIdx.x - seg * a.H), grp = h / (a.H / a.G);
    const int64_t c0 = seg * a.seg_chunks, c1 = c0 + a.seg_chunks < a.chunks ? c0 + a.seg_chunks : a.chunks;
    const int n = (int)(c1 - c0);
    const int64_t bh = (int64_t)b * a.H + h;
    const bool gate = kOut && a.z;

    if (tid == 0) {
        for (uint64_t* bar = &sm.scalars_ready[0]; bar <= &sm.done_yb; ++bar) mbar_init(smem_u32(bar), 1);
        fence_proxy_async();
    }
    if (w == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)), "n"(kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sm.tmem;

    bool late = false;  // a wait gave up: none is tried again, so that the block ends soon
    auto wait = [&](uint64_t* bar, int phase) {
        if (late || mbar_wait(smem_u32(bar), phase & 1)) return;
        late = true;
        atomicOr(&g_device_error_heads, 1u);
    };

    if (w > kIssuer) {
        // the scalars, up to four chunks ahead: a long chain of dependent operations (fp64 sums)
        for (int i = w - kIssuer - 1; i < n; i += 2) {
            if (i > 3) wait(&sm.scalars_free[i & 3], (i - 4) >> 2);
            chunk_scalars<bf16, kTcQ>(sm.s[i & 3], a, b, h, (c0 + i) * kTcQ);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.scalars_ready[i & 3]);
        }
        __syncthreads();
        return;
    }
    if (w == kIssuer) {
        // one lane issues; the warp keeps the barriers.  Once its wait for a copy has given up it starts nothing more.
        bool one = lane == 0;
        auto at = [&](int i) { return (int)((c0 + i) * kTcQ); };
        auto fetch = [&](bf16 (*dst)[kTile], int tiles, const CUtensorMap* map, int row, int i, uint64_t* bar) {
            mbar_expect_tx(smem_u32(bar), tiles * kTile * 2);
            for (int k = 0; k < tiles; ++k) tma_load_4d(smem_u32(dst[k]), map, 64 * k, row, at(i), b, smem_u32(bar));
        };
        if (one) {
            fetch(&sm.x[0], 1, &tm_u, h, 0, &sm.full_x[0]);
            fetch(sm.B[0], HALVES, &tm_B, grp, 0, &sm.full_b[0]);
            if (kOut) fetch(sm.C, HALVES, &tm_C, grp, 0, &sm.full_c);
        }
        for (int i = 0; i < n; ++i) {
            const int buf = i & 1;
            work_sync();                       // the last chunk is done with
            if (one) {
                if (i > 0) mbar_arrive(&sm.scalars_free[(i - 1) & 3]);
                if (kOut) {
                    wait(&sm.full_b[buf], i >> 1);
                    wait(&sm.full_c, i);
                    fence_after();
#pragma unroll
                    for (int k = 0; k < NT / 16; ++k)
                        mma_ss(tmem + kColG, operand(smem_u32(sm.C[k / 4]) + 32 * (k % 4), 16),
                               operand(smem_u32(sm.B[buf][k / 4]) + 32 * (k % 4), 16), instruction(128, 0, 0), k > 0);
                    commit(&sm.done_g);
#pragma unroll
                    for (int k = 0; k < NT / 16; ++k)
                        mma_ss(tmem + kColYa, operand(smem_u32(sm.C[k / 4]) + 32 * (k % 4), 16), operand(smem_u32(sm.S) + 2048 * k, 16),
                               instruction(64, 0, 1), k > 0);
                    commit(&sm.done_ya);
                    if (i > 0) tma_store_4d(&tm_out, 0, h, at(i - 1), b, smem_u32(sm.z));
                }
                if (i + 1 < n) {
                    fetch(&sm.x[buf ^ 1], 1, &tm_u, h, i + 1, &sm.full_x[buf ^ 1]);
                    fetch(sm.B[buf ^ 1], HALVES, &tm_B, grp, i + 1, &sm.full_b[buf ^ 1]);
                }
                if (kOut) {
                    tma_store_wait_read_0();
                    if (gate) fetch(&sm.z, 1, &tm_z, h, i, &sm.full_z);
                    else mbar_arrive(&sm.full_z);
                }
            }
            __syncwarp();
            one = one && !late;
            if (kOut) work_or(0);
            else work_sync();
            if (one) {
                if (!kOut) wait(&sm.full_b[buf], i >> 1);
                fence_after();
                for (int part = 2; part >= 0; --part)
#pragma unroll
                    for (int k = 0; k < kTcQ / 16; ++k)
                        mma_ss(tmem + kColSt, operand(smem_u32(sm.B[buf][0]) + 2048 * k, HALVES == 2 ? kTile * 2 : 0),
                               operand(smem_u32(sm.f[part]) + 2048 * k, 16), instruction(64, 1, 1), part < 2 || k > 0);
                commit(&sm.done_st);
                if (kOut && i + 1 < n) {
                    wait(&sm.done_ya, i);
                    fetch(sm.C, HALVES, &tm_C, grp, i + 1, &sm.full_c);
                }
            }
            __syncwarp();
            if (kOut) {
                work_sync();
                if (one) {
                    fence_after();
#pragma unroll
                    for (int k = 0; k < kTcQ / 16; ++k)
                        mma_ts(tmem + kColYb, tmem + kColM + 8 * k, operand(smem_u32(sm.x[buf]) + 2048 * k, 16), instruction(64, 0, 1), k > 0);
                    commit(&sm.done_yb);
                }
                __syncwarp();
            }
        }
        if (kOut) {
            work_sync();
            if (one) {
                tma_store_4d(&tm_out, 0, h, at(n - 1), b, smem_u32(sm.z));
                tma_store_wait_all();
            }
        }
        // Shared and tensor memory are given up with nothing in flight on them: the last copies and products have
        // been waited for, or are here, and after a wait that gave up each barrier once more.
        if (lane == 0) {
            wait(&sm.full_x[(n - 1) & 1], (n - 1) >> 1);
            if (n > 1) wait(&sm.full_x[n & 1], (n - 2) >> 1);
            wait(&sm.done_st, n - 1);
            if (kOut) {
                wait(&sm.full_z, n - 1);
                wait(&sm.done_yb, n - 1);      // products end in order, so those before it have
            }
            if (late)
                for (uint64_t* bar = &sm.full_x[0]; bar <= &sm.done_yb; ++bar) mbar_drain(smem_u32(bar));
        }
        __syncwarp();
        __syncthreads();
        return;
    }

    const int quarter = w & 3, part4 = w >> 2, r = 32 * quarter + lane;  // this thread's row and quarter of the columns
    const int p0 = 16 * part4;
    const uint32_t tm_row = tmem + ((uint32_t)(32 * quarter) << 16);
    // the state: row n = r, channels p0 .. p0 + 15
    float S[16];
    {
        const float* first = entering_state<kOut>(a, bh, seg);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int p = p0 + k;
            const int64_t at = (int64_t)p * a.N + r;
            S[k] = first && r < a.N && p < a.P &&
                           in_range((a.nseg > 1 ? bh * a.nseg + seg : bh) * a.P * a.N + at, a.nseg > 1 ? states_extent(a) : state_extent(a))
                       ? first[at] : 0.f;
        }
    }
    auto put_state = [&] {  // bf16 S for Ya: row r of [n][p]
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint4 v;
            uint32_t* o = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = Mma<bf16>::pack(S[8 * k + 2 * i], S[8 * k + 2 * i + 1]);
            *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(sm.S) + unit(r, 2 * part4 + k)) = v;
        }
    };
    if (kOut) {
        put_state();
        fence_proxy_async();
    }
    double total = 0.0;

    for (int i = 0; i < n; ++i) {
        const int buf = i & 1;
        const int64_t t0 = (c0 + i) * kTcQ;
        fence_before();
        work_sync();                           // tensor memory, tiles and outputs of the last chunk are done with; S is there
        const auto& sc = sm.s[i & 3];
        wait(&sm.scalars_ready[i & 3], i >> 2);
        wait(&sm.full_x[buf], i >> 1);
        // f U in three parts; values of u that are not finite are noticed on the way
        float probe = 0.f;
        unsigned char* xb = reinterpret_cast<unsigned char*>(sm.x[buf]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int row = (tid >> 3) + 64 * k;
            const uint32_t at = unit(row, tid & 7);
            float v[8];
            widen8(*reinterpret_cast<const uint4*>(xb + at), v);
            const float f = sc.f[row];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (kOut) probe = fmaf(v[e], 0.f, probe);
                v[e] *= f;
            }
#pragma unroll
            for (int part = 0; part < 3; ++part) {
                uint4 o;
                uint32_t* ow = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    ow[e] = Mma<bf16>::pack(v[2 * e], v[2 * e + 1]);
                    v[2 * e] -= __uint_as_float(ow[e] << 16);
                    v[2 * e + 1] -= __uint_as_float(ow[e] & 0xffff0000u);
                }
                *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(sm.f[part]) + at) = o;
            }
        }
        fence_proxy_async();
        int bad = 0;
        if (kOut) bad = work_or(probe != 0.f);
        else work_sync();
        if (kOut && bad) {
            // Such a value would meet the zeros of M above the diagonal: it is left out of the product
            // and its terms are added to the steps that have them, below.
            for (int k = 0; k < 2; ++k) {
                const uint32_t at = unit((tid >> 3) + 64 * k, tid & 7);
                uint32_t* v = reinterpret_cast<uint32_t*>(xb + at);
                for (int e = 0; e < 4; ++e) {
                    if ((v[e] & 0x7f80u) == 0x7f80u) v[e] &= 0xffff0000u;
                    if ((v[e] & 0x7f800000u) == 0x7f800000u) v[e] &= 0xffffu;
                }
            }
            fence_proxy_async();
        }
        if (kOut) {
            // M: row t = r, columns s = 32 part4 .. + 31
            wait(&sm.done_g, i);
            fence_after();
            const float ch = sc.ch[r], cl = sc.cl[r];
            const int s0 = 32 * part4;
            uint32_t m[16];
            if (part4 > quarter) {                     // all above the diagonal
#pragma unroll
                for (int k = 0; k < 16; ++k) m[k] = 0u;
            } else {
                float v[32];
                tmem_load(v, tm_row + kColG + s0);
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const float4 chs = *reinterpret_cast<const float4*>(sc.ch + s0 + k);
                    const float4 cls = *reinterpret_cast<const float4*>(sc.cl + s0 + k);
                    const float4 ws = *reinterpret_cast<const float4*>(sc.w + s0 + k);
                    const float cs[4] = {chs.x, chs.y, chs.z, chs.w}, ls[4] = {cls.x, cls.y, cls.z, cls.w},
                                wv[4] = {ws.x, ws.y, ws.z, ws.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[k + e] = s0 + k + e <= r ? v[k + e] * (ex2((ch - cs[e]) + (cl - ls[e])) * wv[e]) : 0.f;
                    m[k / 2] = Mma<bf16>::pack(v[k], v[k + 1]);
                    m[k / 2 + 1] = Mma<bf16>::pack(v[k + 2], v[k + 3]);
                }
            }
            tmem_store16(tm_row + kColM + s0 / 2, m);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            fence_before();
            work_sync();
        }
        // S' = exp(c_end) S + B^T (f U)
        wait(&sm.done_st, i);
        if (kOut) wait(&sm.done_ya, i);
        fence_after();
        {
            const float dec = ex2(sc.total * kLog2e);
            total += sc.total;
            float v[16];
            tmem_load(v, tm_row + kColSt + p0);
#pragma unroll
            for (int k = 0; k < 16; ++k) S[k] = fmaf(dec, S[k], v[k]);
        }
        if (kOut) {
            put_state();
            wait(&sm.done_yb, i);
            wait(&sm.full_z, i);
            fence_after();
            if (bad) {
                rare_outputs(a, sc, tm_row + kColYa + p0, tm_row + kColYb + p0, reinterpret_cast<unsigned char*>(sm.z), b, h, t0, r, p0);
            } else {
                float ya[16], yb[16];
                tmem_load(ya, tm_row + kColYa + p0);
                tmem_load(yb, tm_row + kColYb + p0);
                const float e = sc.e[r], D = head_param(a, a.D, h);
                unsigned char* zb = reinterpret_cast<unsigned char*>(sm.z);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t at = unit(r, 2 * part4 + k);
                    float xv[8], zv[8], y[8];
                    widen8(*reinterpret_cast<const uint4*>(xb + at), xv);
                    if (gate) widen8(*reinterpret_cast<const uint4*>(zb + at), zv);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        y[j] = fmaf(e, ya[8 * k + j], yb[8 * k + j]);
                        if (a.D) y[j] = fmaf(D, xv[j], y[j]);
                        if (gate) y[j] *= silu(zv[j]);
                    }
                    uint4 o;
                    uint32_t* ow = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
                    for (int j = 0; j < 4; ++j) ow[j] = Mma<bf16>::pack(y[2 * j], y[2 * j + 1]);
                    *reinterpret_cast<uint4*>(zb + at) = o;
                }
            }
            fence_proxy_async();
        }
    }
    // (an infinity or a NaN stays in the state once it is there)
    if (kOut) {
        if (a.h_last && seg == a.nseg - 1 && r < a.N) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (p0 + k < a.P && in_range(bh * a.P * a.N + (int64_t)(p0 + k) * a.N + r, state_extent(a)))
                    a.h_last[bh * a.P * a.N + (int64_t)(p0 + k) * a.N + r] = S[k];
            if (not_finite(S)) segment_by_steps<kOut>(a);
        }
        __syncwarp();
        work_sync();                           // the last chunk's outputs may leave
    } else {
        if (r < a.N) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (p0 + k < a.P && in_range((bh * a.nseg + seg) * a.P * a.N + (int64_t)(p0 + k) * a.N + r, states_extent(a)))
                    a.states[(bh * a.nseg + seg) * a.P * a.N + (int64_t)(p0 + k) * a.N + r] = S[k];
            if (not_finite(S)) segment_by_steps<kOut>(a);
        }
        if (tid == 0 && in_range(bh * a.nseg + seg, segments(a))) a.decays[bh * a.nseg + seg] = (float)total;
    }
    __syncthreads();
    if (w == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kCols));
}

// A wait made to run out of polls, on a barrier that nothing arrives on, and the barrier drained after it.
__global__ void product_probe_kernel(unsigned int polls) {
    __shared__ __align__(8) uint64_t bar;
    mbar_init(smem_u32(&bar), 1);
    fence_proxy_async();
    if (mbar_wait(smem_u32(&bar), 0, polls)) return;
    mbar_drain(smem_u32(&bar));
    atomicOr(&g_device_error_heads, 4u);
}

// A map over (batch, L, heads or groups, width) with boxes of 128 steps by 64 of the width, zeros outside.
bool tc_map(CUtensorMap* m, const void* base, int64_t width, int64_t rows, int64_t L, int64_t batch) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)L, (cuuint64_t)batch};
    const cuuint64_t strides[3] = {(cuuint64_t)width * 2, (cuuint64_t)(width * rows) * 2, (cuuint64_t)(width * rows * L) * 2};
    const cuuint32_t box[4] = {64, 1, kTcQ, 1}, each[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, each,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, bool kOut>
cudaError_t launch(const HeadsArgs& a, cudaStream_t st) {
    CUtensorMap m[5];
    if (!tc_map(&m[0], a.u, a.P, a.H, a.L, a.batch) || !tc_map(&m[1], a.z ? a.z : a.u, a.P, a.H, a.L, a.batch) ||
        !tc_map(&m[2], a.B, a.N, a.G, a.L, a.batch) || !tc_map(&m[3], a.C, a.N, a.G, a.L, a.batch) ||
        !tc_map(&m[4], a.out ? a.out : a.u, a.P, a.H, a.L, a.batch))
        return cudaErrorInvalidValue;
    auto* k = heads_tc_kernel<NT, kOut>;
    constexpr size_t smem = sizeof(TcSmem);
    static_assert(smem <= 227 * 1024, "the tiles of one chunk must fit a block's shared memory");
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    k<<<dim3((unsigned)(a.H * a.nseg), (unsigned)a.batch), kThreads, smem, st>>>(m[0], m[1], m[2], m[3], m[4], a);
    api_count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_heads_tc(const HeadsArgs& a, bool local, cudaStream_t st) {
    if (a.N <= 64) return local ? launch<64, false>(a, st) : launch<64, true>(a, st);
    return local ? launch<128, false>(a, st) : launch<128, true>(a, st);
}

cudaError_t launch_product_probe(unsigned int polls, cudaStream_t st) {
    product_probe_kernel<<<1, 1, 0, st>>>(polls);
    return cudaGetLastError();
}

cudaError_t read_device_error_heads(unsigned int* value, int clear) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error_heads, sizeof(unsigned int));
    if (e == cudaSuccess && clear && *value) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_device_error_heads, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace sscan
