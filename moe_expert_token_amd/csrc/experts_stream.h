// experts_stream.h -- what a wave does where few rows meet an expert's weights
// (library-internal): weights, bf16 or 4-bit with group scales, stream from
// memory straight into registers.
//
//   D[row][feature] = sum over k of X[row][k] * W[feature][k]
//
// v_mfma_f32_16x16x32_bf16 takes 16 rows and 16 features; a lane holds one
// feature (lane & 15) of four rows.  A wave works on four such feature groups
// at once (for the projections two of the gate and the same two of the up
// projection), which share the rows' fragments, and on the chunks of 128 k that
// are its own: the block's waves split k and add their sums through LDS in a
// fixed tree.
//
// A 4-bit value q enters the product as the bf16 number q: as a byte it is the
// e4m3 number q 2^-9, and v_cvt_scalef32_pk_bf16_fp8 makes two bf16 numbers of
// two bytes.  The 8 of q - 8 is taken off by adding the product of the rows
// with -8, which the feature groups share.  So a group's sum is one in fp32
// over terms of up to 15 |x| and of 8 |x|, also where q - 8 is 0, and is scaled
// in fp32 as it is added; an infinite x gives NaN, and so may finite ones whose
// magnitudes in a group sum to 2^128 / 15 or more.  (Signed
// numbers q - 8 need no second term and take longer to make: 45.9 us against
// 39.2, one token, 256 experts of 7168 x 2048, and 1004 against 944, 48 tokens.
// 128 + q from the mantissa's bits, with -136, takes the same time and loses
// four bits more beside a large x.)  The 16 bytes that a lane loads of a weight
// row are 32 neighbouring k; a transpose over the four quarters of the wave
// (two v_permlane32_swap, two v_permlane16_swap) deals them out so that each
// matrix instruction covers 32 neighbouring k, and so one group.
#pragma once

#include <type_traits>

#include "experts.h"

namespace ms {
namespace stream {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kChunk = 128;
constexpr int kGroupsOf16 = 4;  // feature groups of a wave
constexpr int kLongK = 4096;    // from here on eight waves share a sum; below, where each would get few chunks, two
constexpr unsigned kOutside = 0x80000000u;

// Memory of `bytes` bytes that is read a chunk of k at a time; what lies past its end reads as zero.
struct Stream {
    uint64_t p;
    int bytes;

    __device__ __forceinline__ void init(const void* from, int64_t n)
    {
        const uint64_t a = (uint64_t)from;  // the same in every lane
        p = (unsigned)__builtin_amdgcn_readfirstlane((int)a) |
            (uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)(a >> 32)) << 32;
        bytes = __builtin_amdgcn_readfirstlane(n > 0 ? (int)n : 0);
    }
    // The buffer from `skip` bytes on; empty past the end, or unless `any`.
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t from(int skip, bool any) const
    {
        const int left = any && skip < bytes ? bytes - skip : 0;
        return __builtin_amdgcn_make_buffer_rsrc((void*)(p + (unsigned)skip), 0, __builtin_amdgcn_readfirstlane(left),
                                                 0x00020000);
    }
};

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, unsigned at)
{
    return __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
}

// What a wave reads: the weights of its feature groups (group s lies in stream s >> 1, 16 (s & 1) rows of `ld`
// bytes in), their scales (rows of `sld` bytes, in memory or copied to LDS) and the rows.  Group is 0 for bf16
// weights, else the 4-bit weights' group size.  The rows follow each other, or (Picked) lie where `picked` says:
// the bytes from x to this lane's row of each row tile, kOutside where there is none.
template <int Group, bool Picked = false>
struct Source {
    static constexpr bool kPicked = Picked;
    Stream w[2], sc[2], x;
    const char* staged[2];
    int K, chunks;
    unsigned ld, sld, xld;
    unsigned picked[Picked ? 2 : 1];

    __device__ __forceinline__ void init(int k_len)
    {
        K = k_len;
        chunks = (K + kChunk - 1) / kChunk;
        ld = Group ? K / 2 : K * 2;
        sld = Group ? K / (Group ? Group : 1) * 2 : 0;
        xld = K * 2;
    }
    __device__ __forceinline__ void side(int i, const char* rows, const char* scales, int valid)
    {
        w[i].init(rows, (int64_t)min(valid, 32) * ld);
        if (Group) sc[i].init(scales, (int64_t)min(valid, 32) * sld);
    }
};

// Two bytes of 0 .. 15 (the upper two where High) as bf16 numbers: the e4m3 numbers that such bytes stand for, 2^-9 of
// them each (the subnormal ones and the first exponent), times 2^9.
template <bool High>
__device__ __forceinline__ unsigned two_of_e4m3(unsigned v)
{
    return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.0f, High));
}

// 16 rows a group and stream: what a wave has of the weights of one chunk.
template <int Group>
struct Packed {
    u32x4 w[kGroupsOf16][Group ? 1 : 4];
};

// The rows' fragments of a chunk.  As soon as a part of weights or rows is in use, a later chunk's is loaded in its
// place.  Whole: K is a multiple of the chunk, so that only whole chunks are read and a lane's offsets never change.
template <int Group, int RT, bool Whole, bool Staged, class Src = Source<Group>>
struct Chunk {
    u32x4 x[RT][4];

    // 4-bit weights of chunk c
    __device__ __forceinline__ static void load_packed(Packed<Group>& to, const Src& S, int c)
    {
        const int lane = lane_id(), r = lane & 15, q = lane >> 4;
        const bool any = c < S.chunks;
        unsigned at = r * S.ld + q * 16;
        if (!Whole && c * kChunk + q * 32 >= S.K) at = kOutside;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __amdgpu_buffer_rsrc_t b = S.w[i].from(c * (kChunk / 2), any);
            to.w[2 * i][0] = load16(b, at);
            to.w[2 * i + 1][0] = load16(b, at + 16 * S.ld);
        }
    }

    // the scales of a row of group s in chunk c, as bf16 pairs
    __device__ __forceinline__ static void scales_of(const Src& S, int c, int s, unsigned (&to)[2])
    {
        constexpr int G = Group ? Group : 1, kPer = kChunk / G;
        const int r = (lane_id() & 15) + (s & 1) * 16;
        if constexpr (Staged) {
            const char* const row = S.staged[s >> 1] + r * S.sld;
            if constexpr (Whole && Group == 32) {
                const u32x2 v = *(const u32x2*)(row + c * 8);
                to[0] = v[0];
                to[1] = v[1];
            } else if constexpr (Whole && Group == 64) {
                to[0] = *(const unsigned*)(row + c * 4);
            } else {
                // groups past the row's last stand for weights of zero; their scale must be one of the row's own
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int g = min(c * kPer + i, S.K / G - 1);
                    const unsigned v = *(const unsigned short*)(row + 2 * g);
                    to[i >> 1] = i & 1 ? to[i >> 1] | v << 16 : v;
                }
            }
        } else {
            const __amdgpu_buffer_rsrc_t b = S.sc[s >> 1].from(0, true);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int g = min(c * kPer + i, S.K / G - 1);
                const unsigned v = __builtin_amdgcn_raw_buffer_load_b16(b, r * S.sld + 2 * g, 0, 0);
                to[i >> 1] = i & 1 ? to[i >> 1] | v << 16 : v;
            }
        }
    }

    // the 32 k at j of chunk c: fragments, and weights where they are bf16
    __device__ __forceinline__ void load_part(Packed<Group>& to, const Src& S, int c, int j)
    {
        const int lane = lane_id(), r = lane & 15, q = lane >> 4;
        const bool any = c < S.chunks, in = Whole || c * kChunk + j * 32 + q * 8 < S.K;
        if constexpr (Group == 0) {
            const unsigned at = in ? r * S.ld + j * 64 + q * 16 : kOutside;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const __amdgpu_buffer_rsrc_t b = S.w[i].from(c * kChunk * 2, any);
                to.w[2 * i][j] = load16(b, at);
                to.w[2 * i + 1][j] = load16(b, at + 16 * S.ld);
            }
        }
        const __amdgpu_buffer_rsrc_t b = S.x.from(c * kChunk * 2, any);
        if constexpr (Src::kPicked) {  // kOutside has its upper bit and stays outside
#pragma unroll
            for (int t = 0; t < RT; ++t) x[t][j] = load16(b, in ? S.picked[t] + j * 64 + q * 16 : kOutside);
        } else {
            const unsigned at = in ? r * S.xld + j * 64 + q * 16 : kOutside;
#pragma unroll
            for (int t = 0; t < RT; ++t) x[t][j] = load16(b, at + t * 16 * S.xld);
        }
    }

    // Adds chunk c's products to acc, and leaves chunk `next` in its place.
    __device__ __forceinline__ void add_to(f32x4 (&acc)[kGroupsOf16][RT], Packed<Group>& P, const Src& S,
                                           int c, int next)
    {
        if constexpr (Group == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int s = 0; s < kGroupsOf16; ++s)
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        acc[s][t] = mfma_16x16x32(__builtin_bit_cast(bf16x8, x[t][j]),
                                                  __builtin_bit_cast(bf16x8, P.w[s][j]), acc[s][t]);
                load_part(P, S, next, j);
            }
        } else {
            constexpr int kPer = Group / 32;  // matrix instructions a group
            const u32x4 minus8 = {0xc100c100u, 0xc100c100u, 0xc100c100u, 0xc100c100u};
            u32x4 d[kGroupsOf16];
            unsigned now[kGroupsOf16][2];
#pragma unroll
            for (int s = 0; s < kGroupsOf16; ++s) {
                // register j of quarter q <-> register q of quarter j
                const u32x4 w = P.w[s][0];
                const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
                const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
                const auto e = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
                const auto f = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
                d[s] = u32x4{e[0], e[1], f[0], f[1]};
                scales_of(S, c, s, now[s]);
            }
            load_packed(P, S, next);
            __builtin_amdgcn_sched_barrier(0);  // loads go out here, not where the compiler would save registers
#pragma unroll
            for (int j0 = 0; j0 < 4; j0 += kPer) {
                bf16x8 xs[RT][kPer];
                f32x4 base[RT];
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        // k in the order (0, 2), (4, 6), (1, 3), (5, 7) in which the weights' nibbles come apart
                        const u32x4 v = x[t][j0 + j];
                        const u32x4 p = {__builtin_amdgcn_perm(v[1], v[0], 0x05040100),
                                         __builtin_amdgcn_perm(v[3], v[2], 0x05040100),
                                         __builtin_amdgcn_perm(v[1], v[0], 0x07060302),
                                         __builtin_amdgcn_perm(v[3], v[2], 0x07060302)};
                        xs[t][j] = __builtin_bit_cast(bf16x8, p);
                        const f32x4 zero = {0, 0, 0, 0};
                        base[t] = mfma_16x16x32(xs[t][j], __builtin_bit_cast(bf16x8, minus8), j ? base[t] : zero);
                    }
                    load_part(P, S, next, j0 + j);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int s = 0; s < kGroupsOf16; ++s) {
                    f32x4 sum[RT];
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        const unsigned v = d[s][j0 + j], lo = v & 0x0f0f0f0fu, hi = (v >> 4) & 0x0f0f0f0fu;
                        const u32x4 p = {two_of_e4m3<false>(lo), two_of_e4m3<true>(lo), two_of_e4m3<false>(hi),
                                         two_of_e4m3<true>(hi)};
#pragma unroll
                        for (int t = 0; t < RT; ++t)
                            sum[t] = mfma_16x16x32(xs[t][j], __builtin_bit_cast(bf16x8, p), j ? sum[t] : base[t]);
                    }
                    const int g = j0 / kPer;
                    const float f = g & 1 ? bf16_hi(now[s][g >> 1]) : bf16_lo(now[s][g >> 1]);
#pragma unroll
                    for (int t = 0; t < RT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[s][t][i] = fmaf(sum[t][i], f, acc[s][t][i]);
                    if (RT > 2) __builtin_amdgcn_sched_barrier(0);  // keeps the registers of one group apart
                }
            }
        }
    }
};

// How a block's eight waves share its work: KS ways over k, the rest over features; row tiles of up to kRows.
template <int Group, bool Few, int Ways>
struct Split {
    // 64 rows take every register, which groups of 32 leave just enough of; with larger groups they spill (64 rows an
    // expert, 32 experts of 2048 x 2048, groups of 128: 312 us, against 212 in tiles of 32 rows)
    static constexpr int kRows = Few ? 16 : Group == 32 ? 64 : 32;
    static constexpr int KS = Ways;
    static constexpr int FS = kWaves / KS;
    static constexpr int kSums = kWaves * kGroupsOf16 * (kRows / 16) * kWave * 16;  // bytes of the waves' sums
    static constexpr int kStage = kSums > (64 << 10) ? kSums : 64 << 10;             // room for scales, then sums
};

// Copies the scales of a block's features to LDS: side i of feature set f at (2 f + i) * 32 rows, contiguous in memory
// and 64 bytes aligned.  A barrier has to follow.
template <class P, class Src>
__device__ __forceinline__ void stage_scales(char* lds, Src& from, int ks, int fs)
{
    const int side_bytes = 32 * from.sld, t = ks * kWave + lane_id();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        char* const to = lds + (2 * fs + i) * side_bytes;
        from.staged[i] = to;
        const __amdgpu_buffer_rsrc_t b = from.sc[i].from(0, true);
        for (int at = t * 16; at < side_bytes; at += P::KS * kWave * 16) *(u32x4*)(to + at) = load16(b, at);
    }
}

// The sums of RT row tiles by this wave's features over all of its block's ways: total(s, r, f) is that of row r and
// feature f & 15 of group s once the function is back.  `all` is the LDS of the wave's feature set, P::KS * kSet.
template <class P, int RT>
struct Totals {
    static constexpr int kSet = kGroupsOf16 * RT * kWave;  // f32x4 of a wave's sums
    const float* sums;

    // row r, feature f of a group is element r & 3 of lane (f & 15) + 16 (r >> 2 & 3) of row tile r >> 4
    __device__ __forceinline__ float operator()(int s, int r, int f) const
    {
        const int at = ((s * RT + (r >> 4)) * kWave + (f & 15) + 16 * ((r >> 2) & 3)) * 4 + (r & 3);
        float v = 0;
#pragma unroll
        for (int i = 0; i < P::KS; ++i) v += sums[i * kSet * 4 + at];
        return v;
    }
};

template <int Group, class P, int RT, bool Whole, bool Staged, class Src>
__device__ __forceinline__ Totals<P, RT> sum_up(char* lds, const Src& from, int ks, int fs)
{
    constexpr int kSet = Totals<P, RT>::kSet;
    // bf16 rows are read 1 KiB at a time, four chunks, before another wave's turn (340 us against 364 chunk by
    // chunk, four tokens of 4096 x 14336); with 4-bit weights that made no difference
    constexpr int kRun = Group ? 1 : 4;
    const auto after = [](int c) { return (c + 1) % kRun ? c + 1 : c + 1 + (P::KS - 1) * kRun; };
    f32x4 acc[kGroupsOf16][RT];
#pragma unroll
    for (int s = 0; s < kGroupsOf16; ++s)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[s][t] = f32x4{0, 0, 0, 0};
    typedef Chunk<Group, RT, Whole, Staged, Src> C;
    C chunk;
    Packed<Group> weights;
    int c = ks * kRun;
    if constexpr (Group != 0) C::load_packed(weights, from, c);
#pragma unroll
    for (int j = 0; j < 4; ++j) chunk.load_part(weights, from, c, j);
    if (Staged) __syncthreads();
#pragma unroll 1
    while (c < from.chunks) {  // past the last chunk, loads read nothing
        chunk.add_to(acc, weights, from, c, after(c));
        c = after(c);
    }
    if (Staged) __syncthreads();  // the scales' room is the sums'
    f32x4* const all = (f32x4*)lds + (size_t)fs * P::KS * kSet;
#pragma unroll
    for (int s = 0; s < kGroupsOf16; ++s)
#pragma unroll
        for (int t = 0; t < RT; ++t) all[ks * kSet + (s * RT + t) * kWave + lane_id()] = acc[s][t];
    __syncthreads();
    return Totals<P, RT>{(const float*)all};
}

// Whether the scales of a block's features fit the LDS kept for them.
template <int Group, bool Few, int Ways>
bool scales_fit(int K)
{
    typedef Split<Group, Few, Ways> P;
    return (int64_t)64 * P::FS * (K / Group) * 2 <= P::kStage;
}

// h is rounded because it is an operand of the next product (bf16 matrix instructions), y because it is a bf16 output.
__device__ __forceinline__ unsigned short bf16_of(float v) { return (unsigned short)bf16_pack2(v, v); }

}  // namespace stream
}  // namespace ms
