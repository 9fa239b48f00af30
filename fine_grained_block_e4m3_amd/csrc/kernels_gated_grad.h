// kernels_gated_grad.h -- gradient of the gated feed-forward block for gfx950.
//
// Forward: g = X Wg^T, u = X Wu^T, h = act(g) * u.  With dh given:
//   dg = dh * u * act'(g),  du = dh * act(g)              (M, N)
//   dX = dg Wg + du Wu                                    (M, K)
//   dWg = dg^T X,  dWu = du^T X                           (N, K)
// X, Wg, Wu, g, u, dh and the results are BF16; dg and du are formed in FP32
// and rounded once to BF16, the type the matrix instruction takes (every
// product is then exact in FP32 and the sums are FP32).
//
//   1. gated_grad_act_kernel writes dg and du, rows padded with zeros to a
//      multiple of 64 columns (a stream: 6 bytes read, 4 written per element).
//   2. gated_grad_gemm_kernel forms the products, long contractions of few
//      tiles split over workgroups, the last of which joins the FP32 sums.  None of the operands is
//      transposed in memory: an operand whose contraction runs along its rows'
//      elements (dg, du in dX) is staged in LDS as 64-byte row pieces and read
//      with ds_read_b128; one whose contraction runs over its rows (W in dX,
//      dg, du and X in dW) is staged as it lies, 512 contiguous bytes of each
//      of 32 rows, and read with ds_read_b64_tr_b16, which hands each lane
//      four contraction steps of its column.
// What bounds it: the matrix instructions for many rows (and, below their
// rate, the tiles' traffic from L2), the weights and their gradients for few.
// A workgroup of four waves has a 128 x 256 (or 128 x 128) tile and three
// stages of 32 contraction steps; two (three) of them share a compute unit.
// Measured (one MI355X, both kernels): 4096 x 2048 x 7168 434 us (446 on
// a card with a lower clock), 1.16 PFLOP/s in the products at a clock of about
// 1.8 GHz, LDS bank conflicts in the results' pass only, L2 read at 13 TB/s;
// 500 x 2112 x 7168 83-91 us; 64 x 7168 x 7168 114 us (450 MB of operands and
// results: 3.9 TB/s); 256 x 4096 x 7168 107 us; 777 x 500 x 640 17 us.
#pragma once

#include "gated_common.h"
#include "gemm_common.h"

namespace fp8k {

typedef short s16x4 __attribute__((ext_vector_type(4)));

struct GatedGradParams {
    const uint16_t* dh;         // (M, N)
    const uint16_t* g;
    const uint16_t* u;
    const uint16_t* x;          // (M, K)
    const uint16_t* w[2];       // gate, up (N, K)
    uint16_t* d;                // workspace: dg then du, each (M, NP)
    uint16_t* dx;               // (M, K) or null
    uint16_t* dw[2];            // (N, K) or null
    int64_t M, N, K, NP;        // NP: N rounded up to a multiple of 64
    int32_t act;
    int32_t dx_tiles, dw_tiles; // tiles of dX, and of dWg and dWu together
    int32_t dx_splits, dw_splits;   // workgroups per tile along the contraction
    float* dx_part;             // splits > 1: FP32 sums [tile][split] of whole tiles
    float* dw_part;
    int32_t* arrived;           // ... and how many splits of a tile are done: dX's tiles, then the others
    int32_t arrived_tiles;
};

// Eight elements of a row per thread.
template <bool VEC>
__global__ __launch_bounds__(256) void gated_grad_act_kernel(GatedGradParams p) {
    const int64_t per_row = p.NP / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t j = i; j < p.arrived_tiles; j += (int64_t)gridDim.x * 256) p.arrived[j] = 0;
    if (i >= p.M * per_row) return;
    const int64_t m = i / per_row, n = (i - m * per_row) * 8;
    const int64_t at = m * p.N + n;
    i32x4 h{}, g{}, u{};
    if (VEC ? n < p.N : n + 8 <= p.N) {
        // VEC: N % 8 == 0, every row 16-byte aligned
        __builtin_memcpy(&h, VEC ? __builtin_assume_aligned(p.dh + at, 16) : p.dh + at, 16);
        __builtin_memcpy(&g, VEC ? __builtin_assume_aligned(p.g + at, 16) : p.g + at, 16);
        __builtin_memcpy(&u, VEC ? __builtin_assume_aligned(p.u + at, 16) : p.u + at, 16);
    } else if (!VEC) {
        // the row's last elements; the padding stays zero
        for (int j = 0; j < 8 && n + j < p.N; ++j) {
            reinterpret_cast<uint16_t*>(&h)[j] = p.dh[at + j];
            reinterpret_cast<uint16_t*>(&g)[j] = p.g[at + j];
            reinterpret_cast<uint16_t*>(&u)[j] = p.u[at + j];
        }
    }
    i32x4 dg, du;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a[2], b[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t sh = e ? 0 : 16;
            const float hv = __uint_as_float(((uint32_t)h[j] << sh) & 0xFFFF0000u);
            const float gv = __uint_as_float(((uint32_t)g[j] << sh) & 0xFFFF0000u);
            const float uv = __uint_as_float(((uint32_t)u[j] << sh) & 0xFFFF0000u);
            a[e] = hv * uv * gated_act_grad(p.act, gv);
            b[e] = hv * gated_act(p.act, gv);
        }
        dg[j] = (int)pack_bf16x2(a[0], a[1]);
        du[j] = (int)pack_bf16x2(b[0], b[1]);
    }
    i32x4* out = reinterpret_cast<i32x4*>(p.d + m * p.NP + n);
    out[0] = dg;
    out[p.M * p.NP / 8] = du;
}

// PER (2 or 4) wave-wide 16-byte-per-lane loads into consecutive 1 KB pieces of
// LDS from m0 on: piece i from buffer offset voff[i] + soff.
template <int PER>
__device__ __forceinline__ void dma_lds16_run(uint32_t m0, const uint32_t (&voff)[PER], i32x4 rsrc, int soff) {
    static_assert(PER == 2 || PER == 4, "pieces");
    int saved;
    if constexpr (PER == 2)
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                     "buffer_load_dwordx4 %2, %4, %5 offen lds\n\t"
                     "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
                     "buffer_load_dwordx4 %3, %4, %5 offen lds\n\t"
                     "s_mov_b32 m0, %0"
                     : "=&s"(saved) : "s"(m0), "v"(voff[0]), "v"(voff[1]), "s"(rsrc), "s"(soff) : "scc");
    else
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                     "buffer_load_dwordx4 %2, %6, %7 offen lds\n\t"
                     "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
                     "buffer_load_dwordx4 %3, %6, %7 offen lds\n\t"
                     "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
                     "buffer_load_dwordx4 %4, %6, %7 offen lds\n\t"
                     "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
                     "buffer_load_dwordx4 %5, %6, %7 offen lds\n\t"
                     "s_mov_b32 m0, %0"
                     : "=&s"(saved)
                     : "s"(m0), "v"(voff[0]), "v"(voff[1]), "v"(voff[2]), "v"(voff[3]), "s"(rsrc), "s"(soff)
                     : "scc");
}

// One operand of a product in LDS: a stage of 32 contraction steps of BX rows
// of the result (or columns).  SLOW: the contraction runs over the operand's
// memory rows.
//   fast: LDS row of 64 bytes per result row, its four 16-byte chunks at slot
//         chunk ^ (row / 4) % 4 (16 rows at one chunk cover all banks)
//   slow: LDS row of 2 BX bytes per contraction step k, its 32-byte chunks at
//         slot chunk ^ 2 (k % 4) (the 2 x 4 chunks that 32 lanes read cover all banks)
template <int BX, int NWAVES, bool SLOW>
struct GradOperand {
    static constexpr int BYTES = BX * 64;
    static constexpr int PIECES = BYTES / 1024;         // 1 KB wave loads
    static constexpr int PER = PIECES / NWAVES;
    static constexpr int ROWB = 2 * BX;                 // slow: bytes of an LDS row
    static constexpr int KPP = 1024 / ROWB;             // slow: contraction steps per piece
    static_assert(PIECES % NWAVES == 0 && BX >= 128 && BX <= 512, "whole pieces per wave");

    // Byte offset of lane's 16 bytes of piece f from the stage's corner in memory.
    static __device__ __forceinline__ uint32_t source(int f, int lane, uint32_t ld_bytes) {
        if constexpr (SLOW) {
            constexpr int LPK = 64 / KPP;               // lanes per contraction step
            const int k = f * KPP + lane / LPK, pos = lane % LPK;
            const int chunk = (pos >> 1) ^ (2 * (k & 3));
            return (uint32_t)k * ld_bytes + 32 * chunk + 16 * (pos & 1);
        } else {
            const int row = 16 * f + (lane >> 2);
            return (uint32_t)row * ld_bytes + 16 * ((lane & 3) ^ ((lane >> 4) & 3));
        }
    }
    // Per-lane LDS offset of the 32-wide subtile at result row x0 + 32 a.
    static __device__ __forceinline__ uint32_t fragment(int x0, int lane) {
        if constexpr (SLOW) {
            const int t = lane & 15, j = t >> 2, g = lane >> 4;
            const int chunk = (x0 / 16 + (g & 1)) ^ (2 * j);
            return (uint32_t)((8 * (g >> 1) + j) * ROWB + 32 * chunk + 8 * (t & 3));
        } else {
            return (uint32_t)((x0 + (lane & 31)) * 64);
        }
    }
    // Operand of contraction steps 16 s .. 16 s + 15 (s = 0, 1) of a subtile:
    // lane l holds steps 8 (l/32) .. + 7 of result row l%32.
    static __device__ __forceinline__ bf16x8 read(FP8K_LDS const uint8_t* base, uint32_t frag, int s, int lane) {
        if constexpr (SLOW) {
            FP8K_LDS const uint8_t* at = base + frag + s * 16 * ROWB;
            s16x4 v[2];
            v[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FP8K_LDS s16x4*)(at));
            v[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FP8K_LDS s16x4*)(at + 4 * ROWB));
            return __builtin_bit_cast(bf16x8, v);
        } else {
            const uint32_t slot = (uint32_t)((2 * s + (lane >> 5)) ^ ((lane >> 2) & 3)) << 4;
            return __builtin_bit_cast(bf16x8, *(FP8K_LDS const i32x4*)(base + frag + slot));
        }
    }
};

// One BM x BN tile of out (R, S) = sum over segments z of P_z Q_z, P the
// operand of the result's rows and Q of its columns.  Per segment the
// contraction has `len` steps; memory past an operand's end reads as zeros.
struct GradTile {
    const uint16_t* pb[2];      // corner of P and Q at contraction step 0
    const uint16_t* qb[2];
    int64_t p_elems, q_elems;   // elements from the corners to the operands' ends
    int64_t p_ld, q_ld;         // elements between memory rows
    int64_t p_step, q_step;     // elements per contraction step
    int segs;
    int64_t len;
    int split, splits;          // this workgroup's share of the contraction
    uint16_t* out;              // result element (0, 0) of the tile
    float* part;                // splits > 1: the tile's FP32 sums, split by split
    int32_t* arrived;           // ... and its splits that are done
    int64_t out_ld;
    int rows, cols;             // valid part
};

template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES, bool PSLOW>
__device__ __forceinline__ void grad_tile(const GradTile& t, uint8_t* smem) {
    constexpr int NWAVES = WAVES_M * WAVES_N;
    constexpr int TM = BM / WAVES_M, TN = BN / WAVES_N, FI = TM / 32, FJ = TN / 32;
    using P = GradOperand<BM, NWAVES, PSLOW>;
    using Q = GradOperand<BN, NWAVES, true>;
    constexpr int STAGE = P::BYTES + Q::BYTES, NL = P::PER + Q::PER;
    static_assert(STAGES >= 2 && (STAGES - 1) * NL <= 63, "vmcnt range");

    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int wm = wave % WAVES_M, wn = wave / WAVES_M;
    const uint32_t lds0 = uniform((int)lds_addr(smem));
    FP8K_LDS const uint8_t* lds = (FP8K_LDS const uint8_t*)smem;

    // A wave loads PER consecutive 1 KB pieces of each operand.
    uint32_t psrc[P::PER], qsrc[Q::PER];
#pragma unroll
    for (int i = 0; i < P::PER; ++i) psrc[i] = P::source(wave * P::PER + i, lane, (uint32_t)(2 * t.p_ld));
#pragma unroll
    for (int i = 0; i < Q::PER; ++i) qsrc[i] = Q::source(wave * Q::PER + i, lane, (uint32_t)(2 * t.q_ld));
    uint32_t pf[FI], qf[FJ];
#pragma unroll
    for (int a = 0; a < FI; ++a) pf[a] = P::fragment(wm * TM + 32 * a, lane);
#pragma unroll
    for (int b = 0; b < FJ; ++b) qf[b] = Q::fragment(wn * TN + 32 * b, lane);

    const int per_seg = (int)((t.len + 31) / 32);
    const int all = per_seg * t.segs;
    const int first = (int)((int64_t)all * t.split / t.splits);
    const int nblocks = (int)((int64_t)all * (t.split + 1) / t.splits) - first;
    // The blocks come in runs of one buffer resource per operand, along which
    // only the scalar offset advances.  The range check is relied on for the
    // vector offset alone (whether it counts the scalar offset too makes no
    // difference): within a run every row of a block is one of the operand's,
    // and a segment's last block, the only one whose rows may pass the end
    // (t.len is the contraction's own length), is a run of its own with offset
    // 0, so that the resource's range ends exactly at the operand.  Past that,
    // and past the workgroup's blocks, loads read zeros.  Runs are short enough
    // for 32-bit offsets.
    auto range = [](int64_t elems) FP8K_INLINE {
        return (uint32_t)(elems <= 0 ? 0 : elems >= (1ll << 30) ? (1ll << 31) : 2 * elems);
    };
    const int cap = (int)((1ll << 29) / (32 * max(t.p_step, t.q_step)));
    const uint32_t pstep = (uint32_t)(64 * t.p_step), qstep = (uint32_t)(64 * t.q_step);
    i32x4 pr = make_rsrc(t.pb[0], 0u), qr = pr;
    uint32_t poff = 0, qoff = 0;
    int issued = 0, left = 0;
    auto start_run = [&]() FP8K_INLINE {
        const bool live = issued < nblocks;
        const int kb = first + issued;
        const int z = t.segs > 1 && kb >= per_seg ? 1 : 0;
        const int in = kb - z * per_seg;
        const int64_t k0 = (int64_t)in * 32;
        pr = make_rsrc(t.pb[z] + k0 * t.p_step, live ? range(t.p_elems - k0 * t.p_step) : 0u);
        qr = make_rsrc(t.qb[z] + k0 * t.q_step, live ? range(t.q_elems - k0 * t.q_step) : 0u);
        poff = qoff = 0;
        left = !live ? 0x7FFFFFFF : max(1, min(min(per_seg - 1 - in, nblocks - issued), cap));
    };
    auto issue = [&](int stage) FP8K_INLINE {
        if (left == 0) start_run();
        --left;
        ++issued;
        const uint32_t dst = lds0 + (uint32_t)(stage * STAGE);
        dma_lds16_run<P::PER>(dst + (uint32_t)(wave * P::PER * 1024), psrc, pr, (int)poff);
        dma_lds16_run<Q::PER>(dst + (uint32_t)(P::BYTES + wave * Q::PER * 1024), qsrc, qr, (int)qoff);
        poff += pstep;
        qoff += qstep;
    };

    f32x16 acc[FI][FJ];
#pragma unroll
    for (int a = 0; a < FI; ++a)
#pragma unroll
        for (int b = 0; b < FJ; ++b)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.f;

    // Operands are read one half block (16 steps) ahead of the products.  A
    // block's barrier sits in the middle of the block before it: there every
    // wave has read all of its current block, whose stage the loads of the
    // block STAGES further then overwrite, and its own loads of the next
    // block have landed.
#pragma unroll
    for (int s = 0; s < STAGES; ++s) issue(s);
    wait_vmcnt<(STAGES - 1) * NL>();
    lds_barrier();
    struct Operands {
        bf16x8 p[FI], q[FJ];
    };
    auto read = [&](Operands& o, int stage, int s) FP8K_INLINE {
        FP8K_LDS const uint8_t* base = lds + stage * STAGE;
#pragma unroll
        for (int a = 0; a < FI; ++a) o.p[a] = P::read(base, pf[a], s, lane);
#pragma unroll
        for (int b = 0; b < FJ; ++b) o.q[b] = Q::read(base + P::BYTES, qf[b], s, lane);
    };
    auto multiply = [&](const Operands& o) FP8K_INLINE {
#pragma unroll
        for (int a = 0; a < FI; ++a)
#pragma unroll
            for (int b = 0; b < FJ; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(o.q[b], o.p[a], acc[a][b], 0, 0, 0);
    };
    // two reads between one matrix instruction and the next
    auto spread = [&]() FP8K_INLINE {
        static_for<FI * FJ>([&](auto) FP8K_INLINE {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        });
    };
    Operands o0, o1;
    read(o0, 0, 0);
    int stage = 0;
    for (int kb = 0; kb < nblocks; ++kb) {
        const int next = stage + 1 == STAGES ? 0 : stage + 1;
        __builtin_amdgcn_sched_barrier(0);
        read(o1, stage, 1);
        multiply(o0);
        spread();
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wait_vmcnt<(STAGES - 2) * NL>();
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        issue(stage);
        read(o0, next, 0);
        multiply(o1);
        spread();
        stage = next;
    }
    wait_vmcnt<0>();

    // lane l, value v of subtile (a, b): row 32a + l%32, column 32b + 8(v/4) + 4(l/32) + v%4
    const int h = lane >> 5;
    // (tiles of 256 columns are taken only where they fill every slot, unsplit)
    if (BN == 128 && t.splits > 1) {
        // The split that comes last adds all of them, in split order, so that
        // the result does not depend on which one it is.  A thread reads back
        // what the same threads of the other splits wrote.
        // The sums are stored past the caches of an XCD and read the same way (a
        // fence would write back and drop the whole L2: 500 x 2112 x 7168 188
        // us for 92, while that shape was split).
        constexpr int THREADS = 64 * NWAVES, kDeviceScope = 16;
        typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
        const auto sums = __builtin_amdgcn_make_buffer_rsrc(t.part, 0, t.splits * BM * BN * 4, 0x00027000);
        const int own = t.split * (BM * BN * 4);
#pragma unroll
        for (int a = 0; a < FI; ++a)
#pragma unroll
            for (int b = 0; b < FJ; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    __builtin_amdgcn_raw_buffer_store_b128(
                        __builtin_bit_cast(u32x4, f32x4{acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2],
                                                        acc[a][b][4 * q + 3]}),
                        sums, 16 * (int)threadIdx.x, own + ((a * FJ + b) * 4 + q) * 16 * THREADS, kDeviceScope);
        wait_vmcnt<0>();
        __syncthreads();
        int32_t* const before = reinterpret_cast<int32_t*>(smem);   // the stages are done with
        if (threadIdx.x == 0)
            *before = __hip_atomic_fetch_add(t.arrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (uniform(*before) != t.splits - 1) return;
#pragma unroll
        for (int a = 0; a < FI; ++a)
#pragma unroll
            for (int b = 0; b < FJ; ++b)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.f;
        for (int s = 0; s < t.splits; ++s)
#pragma unroll
            for (int a = 0; a < FI; ++a)
#pragma unroll
                for (int b = 0; b < FJ; ++b)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 v = __builtin_bit_cast(
                            f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                       sums, 16 * (int)threadIdx.x,
                                       s * (BM * BN * 4) + ((a * FJ + b) * 4 + q) * 16 * THREADS, kDeviceScope));
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[a][b][4 * q + e] += v[e];
                    }
    }
    // BF16 results through LDS, so that a wave stores whole rows of the tile
    // (straight from the accumulators a store covers 16 bytes of each of 32
    // rows).  Rows of 2 BN + 16 bytes; the stages are done with.
    constexpr int ROW = 2 * BN + 16;
    static_assert(BM * ROW <= STAGES * STAGE, "the tile fits the stages");
    lds_barrier();
#pragma unroll
    for (int a = 0; a < FI; ++a)
#pragma unroll
        for (int b = 0; b < FJ; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint2*>(smem + (wm * TM + 32 * a + (lane & 31)) * ROW +
                                          2 * (wn * TN + 32 * b + 8 * q + 4 * h)) =
                    make_uint2(pack_bf16x2(acc[a][b][4 * q], acc[a][b][4 * q + 1]),
                               pack_bf16x2(acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]));
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    lds_barrier();
    constexpr int LPR = BN / 8, RPW = 64 / LPR;         // lanes per row, rows per wave store
    const int n = 8 * (lane % LPR);
#pragma unroll
    for (int i = 0; i < BM / (RPW * NWAVES); ++i) {
        const int m = (i * NWAVES + wave) * RPW + lane / LPR;
        // K % 128 == 0: whole groups of 8 columns, 16-byte aligned
        if (m < t.rows && n < t.cols)
            *reinterpret_cast<i32x4*>(t.out + (int64_t)m * t.out_ld + n) =
                *reinterpret_cast<const i32x4*>(smem + m * ROW + 2 * n);
    }
}

// Workgroups: the tiles of dX, then those of dWg and dWu (dw_first: the other
// way round, the product with the longer contraction first), each tile's
// splits side by side.
template <int BM, int BNX, int BNW, int WAVES_M, int WAVES_N, int STAGES, int OCC>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N, OCC) void gated_grad_gemm_kernel(GatedGradParams p, bool dw_first) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * (BM + (BNX > BNW ? BNX : BNW)) * 64];
    // workgroup b of a dispatch wave lands on XCD b % 8: each XCD takes a run
    // of consecutive tiles (and shares their operands in its L2)
    auto run_of = [](int b, int count) FP8K_INLINE {
        const int per = count / 8, rest = count % 8, xcd = b % 8;
        return xcd * per + min(xcd, rest) + b / 8;
    };
    const int dx_wgs = p.dx_tiles * p.dx_splits, dw_wgs = p.dw_tiles * p.dw_splits;
    const bool is_dx = dw_first ? (int)blockIdx.x >= dw_wgs : (int)blockIdx.x < dx_wgs;
    const int id = (int)blockIdx.x - (is_dx == dw_first ? (dw_first ? dw_wgs : dx_wgs) : 0);
    int mt, ntile;
    GradTile t;
    t.q_ld = t.q_step = p.K;
    t.out_ld = p.K;
    if (is_dx) {
        const int nt = (int)((p.K + BNX - 1) / BNX);
        const int at = run_of(id, dx_wgs);
        t.splits = p.dx_splits;
        t.split = at % t.splits;
        raster(at / t.splits, (int)((p.M + BM - 1) / BM), nt, 4, mt, ntile);
        const int64_t m0 = (int64_t)mt * BM, n0 = (int64_t)ntile * BNX;
        for (int z = 0; z < 2; ++z) {
            t.pb[z] = p.d + (z * p.M + m0) * p.NP;
            t.qb[z] = p.w[z] + n0;
        }
        t.p_elems = (p.M - m0) * p.NP;
        t.q_elems = p.N * p.K - n0;
        t.p_ld = p.NP;
        t.p_step = 1;
        t.segs = 2;
        t.len = p.N;
        t.out = p.dx + m0 * p.K + n0;
        t.part = p.dx_part + (int64_t)(at / t.splits) * t.splits * (BM * BNX);
        t.arrived = p.arrived + at / t.splits;
        t.rows = (int)min((int64_t)BM, p.M - m0);
        t.cols = (int)min((int64_t)BNX, p.K - n0);
        grad_tile<BM, BNX, WAVES_M, WAVES_N, STAGES, false>(t, smem);
    } else {
        const int nt = (int)((p.K + BNW - 1) / BNW);
        const int rt = (int)((p.N + BM - 1) / BM);
        const int at = run_of(id, dw_wgs);
        t.splits = p.dw_splits;
        t.split = at % t.splits;
        const int tile = at / t.splits;
        const int z = tile >= rt * nt;
        raster(tile - z * rt * nt, rt, nt, 4, mt, ntile);
        const int64_t m0 = (int64_t)mt * BM, n0 = (int64_t)ntile * BNW;
        t.pb[0] = t.pb[1] = p.d + z * p.M * p.NP + m0;
        t.qb[0] = t.qb[1] = p.x + n0;
        t.p_elems = p.M * p.NP - m0;
        t.q_elems = p.M * p.K - n0;
        t.p_ld = t.p_step = p.NP;
        t.segs = 1;
        t.len = p.M;
        t.out = p.dw[z] + m0 * p.K + n0;
        t.part = p.dw_part + (int64_t)tile * t.splits * (BM * BNW);
        t.arrived = p.arrived + (p.dx_splits > 1 ? p.dx_tiles : 0) + tile;
        t.rows = (int)min((int64_t)BM, p.N - m0);
        t.cols = (int)min((int64_t)BNW, p.K - n0);
        grad_tile<BM, BNW, WAVES_M, WAVES_N, STAGES, true>(t, smem);
    }
}

}  // namespace fp8k
