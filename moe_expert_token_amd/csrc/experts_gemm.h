// experts_gemm.h -- the tile product of the experts' matrix kernels
// (library-internal).
//
//   D[row][feature] = sum over k of R[row][k] * F[feature][k]
//
// One block of eight waves makes a tile of 32 MF rows by 256 features (MF up
// to 8: 256 x 256), each wave half of the rows by 64 features, from
// v_mfma_f32_16x16x32_bf16 with the features as its rows, so that a lane ends
// with four neighbouring features of one row.  An operand comes in one of two
// orders: k-contiguous (rows of a matrix), or k-strided (its columns), where
// the transposing LDS read turns [k][16] blocks into fragments on the way.
//
// The tile of 64 k is loaded straight into LDS (16 bytes a lane, no
// registers), two tiles deep (128 KiB).  Rows, features and k past the
// operand's end are loads out of the buffer descriptor's range: they read as
// zero and touch no memory.
#pragma once

#include "experts.h"

namespace ms {

constexpr int kGemmThreads = 512;
constexpr int kTileK = 64;
constexpr int kTileFeatures = 256;
constexpr int kTileRows = 256;
constexpr int kOperandBytes = 256 * kTileK * 2;  // 32 KiB of LDS an operand and stage
constexpr int kGemmLds = 4 * kOperandBytes;

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr unsigned kOutside = 0x80000000u;  // an offset that no descriptor here reaches

// N loads of 16 bytes a lane from `rsrc`, at voff[i], into LDS at `lds` + 8192 i (the wave's first byte; lane l's
// land 16 l further).  In assembly so that the compiler does not take each later LDS read for one of this tile and
// wait for it: the loads of a tile are waited for once, by wait_loads() and the barrier in front of its first read.
// It has no register output, and nothing else in the kernels that use it goes by m0.  The waits inside are those
// the hardware asks for: five states after a descriptor's word came from a vector instruction, one after m0 changed.
template <int N>
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, unsigned lds, const unsigned (&voff)[N])
{
    static_assert(N >= 1 && N <= 4, "tiles of at most 256 rows");
    if constexpr (N == 1)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds"
                     :
                     : "s"(lds), "s"(rsrc), "v"(voff[0])
                     : "memory", "scc");
    else if constexpr (N == 2)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds\n\t"
                     "s_add_u32 m0, %0, 0x2000\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %1, 0 offen lds"
                     :
                     : "s"(lds), "s"(rsrc), "v"(voff[0]), "v"(voff[1])
                     : "memory", "scc");
    else if constexpr (N == 3)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds\n\t"
                     "s_add_u32 m0, %0, 0x2000\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %1, 0 offen lds\n\t"
                     "s_add_u32 m0, %0, 0x4000\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, %1, 0 offen lds"
                     :
                     : "s"(lds), "s"(rsrc), "v"(voff[0]), "v"(voff[1]), "v"(voff[2])
                     : "memory", "scc");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds\n\t"
                     "s_add_u32 m0, %0, 0x2000\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %1, 0 offen lds\n\t"
                     "s_add_u32 m0, %0, 0x4000\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, %1, 0 offen lds\n\t"
                     "s_add_u32 m0, %0, 0x6000\n\ts_nop 0\n\tbuffer_load_dwordx4 %5, %1, 0 offen lds"
                     :
                     : "s"(lds), "s"(rsrc), "v"(voff[0]), "v"(voff[1]), "v"(voff[2]), "v"(voff[3])
                     : "memory", "scc");
}

__device__ __forceinline__ u32x4 buffer_of(const char* p, unsigned bytes)
{
    const uint64_t a = (uint64_t)p;
    return u32x4{(unsigned)a, (unsigned)(a >> 32) & 0xffffu, bytes, 0x00020000u};
}

__device__ __forceinline__ unsigned lds_offset(const void* p) { return (unsigned)(uintptr_t)(lds_void*)p; }

// s_waitcnt vmcnt(0): everything this wave has loaded (into LDS too) is there.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }

// An operand whose rows (or features) run along memory rows of k.
//   LDS: [256][64] bf16; the 16-byte piece c of row r lies at piece c ^ (r & 7), so that the eight lanes of a
//   fragment read that are served together fall on all banks.
struct KContiguous {
    static constexpr int kReads = 1;  // LDS instructions a fragment
    const char* p;     // (row 0, k 0)
    unsigned ld;       // bytes from row to row
    unsigned bytes;    // from p to the end of the last valid row
    int K;
    unsigned voff;     // this thread's first piece
    unsigned next;     // bytes to the same piece of the next instruction's rows
    int piece8;        // its k within the tile

    // LDS rows 64 i + r hold the operand's rows `stride` * i + row: in order for stride 64 and row = r.
    __device__ __forceinline__ void init(const void* base, int ld_elems, int valid_rows, int k_len, int stride, int row)
    {
        p = (const char*)base;
        ld = (unsigned)ld_elems * 2;
        bytes = (unsigned)valid_rows * ld;
        K = k_len;
        const int t = threadIdx.x, r = t >> 3, c = (t & 7) ^ (r & 7);
        piece8 = c * 8;
        voff = (unsigned)row * ld + (unsigned)c * 16;
        next = (unsigned)stride * ld;
    }
    __device__ __forceinline__ void init(const void* base, int ld_elems, int valid_rows, int k_len)
    {
        init(base, ld_elems, valid_rows, k_len, 64, threadIdx.x >> 3);
    }

    // Starts the loads of tile kt into LDS at `lds`: N instructions of 64 rows.
    template <int N>
    __device__ __forceinline__ void load(int kt, unsigned lds) const
    {
        const int k0 = kt * kTileK;
        const bool any = k0 < K;
        const unsigned skip = any ? (unsigned)k0 * 2 : 0;
        unsigned v[N];
        v[0] = k0 + piece8 < K ? voff : kOutside;
#pragma unroll
        for (int i = 1; i < N; ++i) v[i] = v[i - 1] + next;
        load_to_lds<N>(buffer_of(p + skip, any ? bytes - skip : 0), lds + wave_id() * 1024, v);
    }

    // The fragment of rows `row0` .. + 16 and k half `half`: lane & 15 the row, 8 (lane >> 4) the k.
    static __device__ __forceinline__ bf16x8 fragment(const char* lds, int row0, int half)
    {
        const int lane = lane_id(), r = lane & 15, c = (half * 4 + (lane >> 4)) ^ (r & 7);
        return *(const bf16x8*)(lds + (row0 + r) * 128 + c * 16);
    }
};

// An operand whose k runs along memory rows of features.
//   LDS: [64][256] bf16; the 32-byte piece c of row k lies at piece c ^ (k & 3 | (k >> 3 & 3) << 2): the sixteen
//   rows of a transposing read (four of every eight) fall on different banks.
struct KStrided {
    static constexpr int kReads = 2;
    const char* p;     // (k 0, feature 0 of the tile)
    unsigned ld;       // bytes from k to k + 1
    int K;
    unsigned voff[2];  // of even and odd instructions

    __device__ __forceinline__ void init(const void* base, int ld_elems, int valid_features, int k_len)
    {
        p = (const char*)base;
        ld = (unsigned)ld_elems * 2;
        K = k_len;
        const int t = threadIdx.x, r = t >> 5;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = (t & 31) ^ ((r & 3) << 1) ^ ((r >> 3) << 3) ^ (i << 4);
            voff[i] = c * 8 < valid_features ? (unsigned)r * ld + (unsigned)c * 16 : kOutside;
        }
    }

    // 16 rows of k an instruction; all 256 features whatever N.
    template <int N>
    __device__ __forceinline__ void load(int kt, unsigned lds) const
    {
        const int left = K - kt * kTileK;
        const bool any = left > 0;
        const unsigned v[4] = {voff[0], voff[1] + 16 * ld, voff[0] + 32 * ld, voff[1] + 48 * ld};
        load_to_lds<4>(buffer_of(p + (any ? (int64_t)kt * kTileK * ld : 0), any ? (unsigned)min(left, kTileK) * ld : 0),
                       lds + wave_id() * 1024, v);
    }

    static __device__ __forceinline__ bf16x8 fragment(const char* lds, int f0, int half)
    {
        // lanes 4 r .. 4 r + 3 of each sixteen name row r of a [4][16] block; the block comes back by columns
        const int lane = lane_id(), b = lane >> 4, r = (lane >> 2) & 3, j = lane & 3;
        const int k = half * 32 + b * 8 + r;
        const int piece = (f0 >> 4) ^ (r | (b << 2));
        const char* at = lds + k * 512 + piece * 32 + j * 8;
        union {
            s16x4 h[2];
            bf16x8 v;
        } u;
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * 512));
        return u.v;
    }
};

// Asks for `Reads` LDS reads spread among `Products` matrix instructions, so that both proceed.
template <int Reads, int Products, int I = 0>
__device__ __forceinline__ void interleave()
{
    if constexpr (I < Reads) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, (I + 1) * Products / Reads - I * Products / Reads, 0);
        interleave<Reads, Products, I + 1>();
    }
}

template <int MF>
using Acc = f32x4[MF][4];

// acc[m][f]: rows 16 (MF wr + m) + (lane & 15), features 64 wf + 16 f + 4 (lane >> 4) .. + 4 of the tile, with
// wr = wave >> 2, wf = wave & 3.  `lds`: kGemmLds bytes.  Ends with a barrier: LDS is free.
template <int MF, class R, class F>
__device__ __forceinline__ void tile_product(const R& r, const F& f, int K, char* lds, Acc<MF>& acc)
{
    const int wr = wave_id() >> 2, wf = wave_id() & 3, nk = (K + kTileK - 1) / kTileK;
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
    const unsigned base = __builtin_amdgcn_readfirstlane(lds_offset(lds));
    const auto start = [&](int kt) {
        const unsigned at = base + (kt & 1) * 2 * kOperandBytes;
        r.template load<(MF + 1) / 2>(kt, at);
        f.template load<4>(kt, at + kOperandBytes);
    };
    bf16x8 ra[2][MF], fa[2][4];
    const auto fragments = [&](int kt, int half) {
        const char* const at = lds + (kt & 1) * 2 * kOperandBytes;
#pragma unroll
        for (int n = 0; n < 4; ++n) fa[half][n] = F::fragment(at + kOperandBytes, wf * 64 + n * 16, half);
#pragma unroll
        for (int m = 0; m < MF; ++m) ra[half][m] = R::fragment(at, (wr * MF + m) * 16, half);
    };
    const auto multiply = [&](int half) {
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n) acc[m][n] = mfma_16x16x32(fa[half][n], ra[half][m], acc[m][n]);
    };
    if (nk > 0) {
        start(0);
        start(1);
        wait_loads();
        __syncthreads();
        fragments(0, 0);
        for (int kt = 0; kt < nk; ++kt) {
            fragments(kt, 1);
            multiply(0);
            interleave<MF * R::kReads + 4 * F::kReads, 4 * MF>();
            wait_loads();
            __syncthreads();
            start(kt + 2);
            fragments(kt + 1, 0);
            multiply(1);
            interleave<MF * R::kReads + 4 * F::kReads, 4 * MF>();
        }
        wait_loads();
        __syncthreads();
    }
}

}  // namespace ms
