// experts_tiles.h -- from the tile product of experts_gemm.h to rows in memory,
// and which block makes which tile (library-internal).
#pragma once

#include "experts_gemm.h"

namespace ms {

// ---- from accumulators to rows ----

__device__ __forceinline__ u32x2 pack4(f32x4 v) { return u32x2{bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3])}; }

// A staged output tile: rows of `Bytes` bytes in LDS, their 16-byte pieces permuted by the row so that the sixteen
// rows a wave writes at once spread over the banks; from there rows go out whole.
template <int Bytes>
struct Stage {
    static __device__ __forceinline__ char* at(char* lds, int row, int byte)
    {
        return lds + row * Bytes + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15);
    }

    // Rows [0, nr) of at most 32 MF and bytes [0, valid) of the tile to out + row * ld; Vec divides valid and the
    // rows' alignment.
    template <class Vec, int MF>
    static __device__ __forceinline__ void store(const char* lds, int nr, int valid, char* out, int64_t ld)
    {
        constexpr int kLanes = Bytes / (int)sizeof(Vec), kRows = kGemmThreads / kLanes;
        constexpr int kTurns = (32 * MF + kRows - 1) / kRows, kBatch = kTurns < 4 ? kTurns : 4;
        const int b = (int)(threadIdx.x % kLanes) * (int)sizeof(Vec), r0 = threadIdx.x / kLanes;
        if (b >= valid) return;
#pragma unroll
        for (int t = 0; t < kTurns; t += kBatch) {
            Vec v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                v[i] = *(const Vec*)at((char*)lds, min(r0 + (t + i) * kRows, 32 * MF - 1), b);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = r0 + (t + i) * kRows;
                if (r < nr) *(Vec*)(out + r * ld + b) = v[i];
            }
        }
    }
};

// The block's place among `tiles` x `across`: chunks of 32 neighbouring places go to one XCD (blocks are dealt to
// the eight in turn), and within a chunk four row tiles meet eight feature tiles, so its L2 sees each operand
// tile several times at once.
struct Place {
    int tile, across;
};
__device__ __forceinline__ Place place_of(const GridSpan& g, int across)
{
    const int b = span_block(g), slot = b >> 3, i = ((slot >> 5) * 8 + (b & 7)) * 32 + (slot & 31);
    const int group = i / (4 * across), rest = i - group * 4 * across;
    return Place{group * 4 + (rest & 3), rest >> 2};
}

// Blocks that cover tiles x across under place_of.
inline int64_t places(int64_t tiles, int across) { return ((tiles + 3) / 4 * 4 * across + 255) / 256 * 256; }

// Calls f with the fragment rows (1 .. 8, or Small 1 .. 2) that cover nr rows as a constant.
template <bool Small, class F>
__device__ __forceinline__ void with_rows(int nr, F&& f)
{
    if constexpr (Small) {
        if (nr <= 32) f(std::integral_constant<int, 1>());
        else f(std::integral_constant<int, 2>());
    } else switch ((nr + 31) >> 5) {
        case 1: f(std::integral_constant<int, 1>()); break;
        case 2: f(std::integral_constant<int, 2>()); break;
        case 3: f(std::integral_constant<int, 3>()); break;
        case 4: f(std::integral_constant<int, 4>()); break;
        case 5: f(std::integral_constant<int, 5>()); break;
        case 6: f(std::integral_constant<int, 6>()); break;
        case 7: f(std::integral_constant<int, 7>()); break;
        default: f(std::integral_constant<int, 8>()); break;
    }
}

// The slots of nr rows of `width` elements from `first`.
template <int MF>
__device__ __forceinline__ void row_slots(KContiguous& r, const char* first, int width, int nr)
{
    constexpr int kFirst = 32 * low_rows(MF);
    r.slot(0, first, min(nr, kFirst));
    r.slot(1, first + (int64_t)kFirst * width * 2, nr - kFirst);
}

typedef Stage<kTileFeatures * 2> WideStage;

// The packed values of each (m, n) to rows of `out`.
template <int MF, class Value>
__device__ __forceinline__ void write_tile(char* lds, int nr, int valid, char* out, int64_t ld, Value value)
{
    const int lane = lane_id();
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int row = row_of<MF>(m) + (lane & 15), c = feature_of(n) + 4 * (lane >> 4);
            *(u32x2*)WideStage::at(lds, row, 2 * c) = value(m, n);
        }
    __syncthreads();
    WideStage::store<u32x4, MF>(lds, nr, 2 * valid, out, ld);
}

}  // namespace ms
