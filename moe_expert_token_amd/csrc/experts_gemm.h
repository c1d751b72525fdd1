// experts_gemm.h -- the tile product of the experts' matrix kernels
// (library-internal).
//
//   D[row][feature] = sum over k of R[row][k] * F[feature][k]
//
// One block of eight waves makes a tile of 32 MF rows by 256 features (MF up
// to 8: 256 x 256) from v_mfma_f32_16x16x32_bf16, with the features as its
// rows, so that a lane ends with four neighbouring features of one row.  An
// operand comes in one of two orders: k-contiguous (rows of a matrix), or
// k-strided (its columns), where the transposing LDS read turns [k][16] blocks
// into fragments on the way.
//
// A tile of 64 k is four slots of LDS, the halves R0, R1 of the rows and F0, F1
// of the features, 16 KiB each, loaded straight into LDS (16 bytes a lane, no
// registers); two tiles fit (128 KiB).  A step over tile t has four phases,
// one barrier each:
//
//   product   R0 F0       R0 F1       R1 F1       R1 F0
//   reads     F1 (t)      R1 (t)      R0 (t+1)    F0 (t+1)    fragments for the next phase
//   loads     F0 (t+2)    F1 (t+2)    R1 (t+2)    R0 (t+3)    into the slot read a phase ago
//
// A slot is free as soon as its fragments are in registers, so its next load
// starts seven phases before it is read: that is what hides the memory's
// latency.  (With loads one step ahead, grad_xe of 32 experts of 7168 x 2048
// ran at 1.12 PFLOP/s, and at 1.45 with the loads left out.)
//
// Weight gradients of 8 experts of 1024 rows, 4096 x 14336, take 33 us a tile
// on average.  Cut to one step of k they take 10.6: so 1.5 us a step, 1.43
// PFLOP/s over 256 CUs, and a third of the time is the start and the end of
// tiles; without the stores the whole takes 1066 us instead of 1393.
//
// Rows, features and k past the operand's end are loads out of the buffer
// descriptor's range: they read as zero and touch no memory.
#pragma once

#include <type_traits>

#include "experts.h"

namespace ms {

constexpr int kGemmThreads = 512;
constexpr int kTileK = 64;
constexpr int kTileFeatures = 256;
constexpr int kTileRows = 256;
constexpr int kSlot = 128 * kTileK * 2;  // 16 KiB

// The LDS of a product.  Where the experts have few rows, a tile of 64 (Small) needs one slot of 8 KiB for them, so
// that two blocks fit a CU: with nothing but weights to wait for, that is what counts.
template <bool Small>
struct Lds {
    static constexpr int kRows = Small ? 64 : kTileRows;
    static constexpr int kFeatures = Small ? kSlot / 2 : 2 * kSlot;  // where F0 lies in a tile
    static constexpr int kTile = kFeatures + 2 * kSlot;
    static constexpr int kBytes = 2 * kTile;
};

// Row fragments of a wave in R0, of MF in all; R1 has the others.
constexpr int low_rows(int MF) { return MF <= 2 ? MF : (MF + 1) / 2; }

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr unsigned kOutside = 0x80000000u;  // an offset that no descriptor here reaches

// A load of 16 bytes a lane from `rsrc` at voff into LDS at `lds` (the wave's first byte; lane l's land 16 l
// further).  In assembly so that the compiler does not take each later LDS read for one of this slot and wait for
// it: a slot is waited for once, by wait_loads() and the barrier in front of the phase that reads it.  It has no
// register output, and nothing else in the kernels that use it goes by m0.  The wait inside is the one the
// hardware asks for: five states after a descriptor's word came from a vector instruction (one after m0 changed).
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, unsigned lds, unsigned voff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds"
                 :
                 : "s"(lds), "s"(rsrc), "v"(voff));
}

__device__ __forceinline__ u32x4 buffer_of(const char* p, unsigned bytes)
{
    const uint64_t a = (uint64_t)p;
    // the same in every lane; the reads put into scalar registers what the compiler computed in vector ones
    return u32x4{(unsigned)__builtin_amdgcn_readfirstlane((int)a),
                 (unsigned)__builtin_amdgcn_readfirstlane((int)(a >> 32)) & 0xffffu,
                 (unsigned)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}

__device__ __forceinline__ unsigned lds_offset(const void* p) { return (unsigned)(uintptr_t)(lds_void*)p; }

// Waits until all but this wave's last N loads have landed (those into LDS too).
template <int N>
__device__ __forceinline__ void wait_loads()
{
    static_assert(N < 64, "six bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4 << 14) | 0x0f70);
}

// An operand whose rows (or features) run along memory rows of k.
//   LDS: [128][64] bf16 a slot; the 16-byte piece c of row r lies at piece c ^ (r & 7), so that the eight lanes of
//   a fragment read that are served together fall on all banks.
struct KContiguous {
    static constexpr bool kTransposed = false;
    const char* p[2];   // of each slot: (row 0, k 0)
    unsigned bytes[2];  // from p to the end of the slot's last valid row
    unsigned ld;        // bytes from row to row
    int K;
    unsigned voff;      // this thread's first piece
    int piece8;         // its k within the tile

    __device__ __forceinline__ void init(int ld_elems, int k_len)
    {
        ld = (unsigned)ld_elems * 2;
        K = k_len;
        const int t = threadIdx.x, r = t >> 3, c = (t & 7) ^ (r & 7);
        piece8 = c * 8;
        voff = (unsigned)r * ld + (unsigned)c * 16;
    }
    // The first of slot s's rows, and how many there are (none or fewer: the slot is zero).
    __device__ __forceinline__ void slot(int s, const char* first, int valid)
    {
        p[s] = first;
        bytes[s] = (unsigned)max(0, min(valid, 128)) * ld;
    }

    // Starts the loads of slot s of tile kt: N of 64 rows.
    template <int N>
    __device__ __forceinline__ void load(int s, int kt, unsigned lds) const
    {
        const int k0 = kt * kTileK, skip = k0 < K ? k0 * 2 : 0x7fffffff;
        const u32x4 rsrc = buffer_of(p[s] + (unsigned)k0 * 2u, (unsigned)max((int)bytes[s] - skip, 0));
        const unsigned v = k0 + piece8 < K ? voff : kOutside;
#pragma unroll
        for (int i = 0; i < N; ++i) load_to_lds(rsrc, lds + wave_id() * 1024 + i * 8192, v + i * 64 * ld);
    }

    // The fragment of the slot's rows `row0` .. + 16 and k half `half`: lane & 15 the row, 8 (lane >> 4) the k.
    static __device__ __forceinline__ bf16x8 fragment(const char* lds, int row0, int half)
    {
        const int lane = lane_id(), r = lane & 15, c = (half * 4 + (lane >> 4)) ^ (r & 7);
        return *(const bf16x8*)(lds + (row0 + r) * 128 + c * 16);
    }
};

// An operand whose k runs along memory rows of features.
//   LDS: [64][128] bf16 a slot; the 32-byte piece c of row k lies at piece c ^ (k & 3 | (k >> 3 & 1) << 2): the
//   eight rows that a transposing read is served at once fall on different banks.
struct KStrided {
    static constexpr bool kTransposed = true;
    const char* p[2];  // of each slot: (k 0, feature 0)
    unsigned voff[2];  // of this thread's piece; kOutside past the slot's features
    unsigned ld;       // bytes from k to k + 1
    int K;

    __device__ __forceinline__ void init(int ld_elems, int k_len)
    {
        ld = (unsigned)ld_elems * 2;
        K = k_len;
    }
    __device__ __forceinline__ void slot(int s, const char* first, int valid)
    {
        p[s] = first;
        const int t = threadIdx.x, r = t >> 4, c = (t & 15) ^ ((r & 3) << 1) ^ (((r >> 3) & 1) << 3);
        voff[s] = c * 8 < valid ? (unsigned)r * ld + (unsigned)c * 16 : kOutside;
    }

    // Starts the loads of slot s of tile kt: two of 32 rows of k.
    template <int N>
    __device__ __forceinline__ void load(int s, int kt, unsigned lds) const
    {
        static_assert(N == 2, "64 rows of k");
        const int rows = min(max(K - kt * kTileK, 0), kTileK);
        const u32x4 rsrc = buffer_of(p[s] + (int64_t)kt * kTileK * ld, (unsigned)rows * ld);
#pragma unroll
        for (int i = 0; i < 2; ++i) load_to_lds(rsrc, lds + wave_id() * 1024 + i * 8192, voff[s] + i * 32 * ld);
    }

    static __device__ __forceinline__ bf16x8 fragment(const char* lds, int f0, int half)
    {
        // lanes 4 r .. 4 r + 3 of each sixteen name row r of a [4][16] block; the block comes back by columns
        const int lane = lane_id(), b = lane >> 4, r = (lane >> 2) & 3, j = lane & 3;
        const int k = half * 32 + b * 8 + r;
        const int piece = (f0 >> 4) ^ (r | ((b & 1) << 2));
        const char* at = lds + k * 256 + piece * 32 + j * 8;
        union {
            s16x4 h[2];
            bf16x8 v;
        } u;
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * 256));
        return u.v;
    }
};

template <int MF>
using Acc = f32x4[MF][4];

// Where acc[m][n] of this wave lies in the tile: rows row_of<MF>(m) + (lane & 15), features feature_of(n) +
// 4 (lane >> 4) .. + 4.  Slot R0 holds the first 32 low_rows(MF) rows, R1 the rest.
template <int MF>
__device__ __forceinline__ int row_of(int m)
{
    constexpr int A = low_rows(MF), B = MF - A;
    const int wr = wave_id() >> 2;
    return m < A ? 16 * (A * wr + m) : 32 * A + 16 * (B * wr + m - A);
}
__device__ __forceinline__ int feature_of(int n) { return (n >> 1) * 128 + 32 * (wave_id() & 3) + 16 * (n & 1); }

// The tile's product.  `lds`: Lds<Small>::kBytes.  Ends with a barrier: LDS is free.
template <bool Small, int MF, class R, class F>
__device__ __forceinline__ void tile_product(const R& r, const F& f, int K, char* lds, Acc<MF>& acc)
{
    constexpr int A = low_rows(MF), B = MF - A;  // row fragments of a wave in R0 and R1
    constexpr int kTile = Lds<Small>::kTile, kFeatures = Lds<Small>::kFeatures;
    static_assert(!Small || B == 0, "no slot for R1");
    constexpr int a = R::kTransposed ? 2 : (A + 1) / 2, b = R::kTransposed ? 2 : (B + 1) / 2;  // loads of R0 and R1
    const int wr = wave_id() >> 2, wf = wave_id() & 3, nk = (K + kTileK - 1) / kTileK;
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
    if (nk == 0) return;
    const unsigned base = __builtin_amdgcn_readfirstlane(lds_offset(lds));
    // slots of a tile: R0, R1, F0, F1
    const auto load_r = [&](int s, int kt) {
        const unsigned at = base + (kt & 1) * kTile + s * kSlot;
        if (s == 0) r.template load<a>(0, kt, at);
        else r.template load<b>(1, kt, at);
    };
    const auto load_f = [&](int s, int kt) { f.template load<2>(s, kt, base + (kt & 1) * kTile + kFeatures + s * kSlot); };
    bf16x8 r0[A][2], r1[B ? B : 1][2], fx[2][2], fy[2][2];
    const auto read_r0 = [&](int kt, int i) {
        r0[i >> 1][i & 1] = R::fragment(lds + (kt & 1) * kTile, 16 * (A * wr + (i >> 1)), i & 1);
    };
    const auto read_r1 = [&](int kt, int i) {
        r1[i >> 1][i & 1] = R::fragment(lds + (kt & 1) * kTile + kSlot, 16 * (B * wr + (i >> 1)), i & 1);
    };
    const auto read_f = [&](bf16x8 (&to)[2][2], int s, int kt, int i) {
        to[i >> 1][i & 1] = F::fragment(lds + (kt & 1) * kTile + kFeatures + s * kSlot, 32 * wf + 16 * (i >> 1), i & 1);
    };
    // One phase: products of `count` row fragments with two feature fragments; the `reads` LDS reads of the next
    // phase go out in the first half of the products, the loads in their middle.
    const auto phase = [&](auto count, auto first, auto side, const bf16x8 (*rows)[2], const bf16x8 (&feat)[2][2],
                           auto reads, auto read, auto load, auto newer) {
        constexpr int C = decltype(count)::value, M0 = decltype(first)::value, N0 = decltype(side)::value * 2;
        constexpr int kReads = decltype(reads)::value, kChunks = C > 0 ? C : 1, kOver = (kChunks + 1) / 2;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
#pragma unroll
            for (int i = 0; i < kReads; ++i)
                if (i * kOver / (kReads ? kReads : 1) == c) read(i);
            if (c == kChunks / 2) load();
            if constexpr (C > 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
                        acc[M0 + c][N0 + n] = mfma_16x16x32(feat[n][h], rows[c][h], acc[M0 + c][N0 + n]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_loads<decltype(newer)::value>();
        __syncthreads();
    };
#define MS_INT(x) std::integral_constant<int, (x)>()
    const auto step = [&](int kt, bf16x8 (&f0)[2][2], bf16x8 (&f1)[2][2]) {
        phase(MS_INT(A), MS_INT(0), MS_INT(0), r0, f0, MS_INT(4), [&](int i) { read_f(f1, 1, kt, i); },
              [&] { load_f(0, kt + 2); }, MS_INT(2 * a + b + 6));
        phase(MS_INT(A), MS_INT(0), MS_INT(1), r0, f1, MS_INT(2 * B), [&](int i) { read_r1(kt, i); },
              [&] { load_f(1, kt + 2); }, MS_INT(a + b + 8));
        phase(MS_INT(B), MS_INT(A), MS_INT(1), r1, f1, MS_INT(2 * A), [&](int i) { read_r0(kt + 1, i); },
              [&] { load_r(1, kt + 2); }, MS_INT(a + 2 * b + 6));
        phase(MS_INT(B), MS_INT(A), MS_INT(0), r1, f0, MS_INT(4), [&](int i) { read_f(f1, 0, kt + 1, i); },
              [&] { load_r(0, kt + 3); }, MS_INT(2 * a + 2 * b + 4));
    };
#undef MS_INT
    // in the steps' order, so that what a wait counts as newer is the same from the first phase on
    for (int kt = 0; kt < 2; ++kt) {
        load_r(0, kt);
        load_f(0, kt);
        load_f(1, kt);
        load_r(1, kt);
    }
    wait_loads<a + 2 * b + 6>();  // R0 and F0
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2 * A; ++i) read_r0(0, i);
#pragma unroll
    for (int i = 0; i < 4; ++i) read_f(fx, 0, 0, i);
    wait_loads<a + 2 * b + 4>();  // F1
    __syncthreads();
    load_r(0, 2);
    for (int kt = 0;;) {
        step(kt, fx, fy);
        if (++kt >= nk) break;
        step(kt, fy, fx);
        if (++kt >= nk) break;
    }
    wait_loads<0>();
    __syncthreads();
}

}  // namespace ms
