// experts_ffn.hip -- the matrix products of the experts' gated block, a row tile of one expert by a tile of features a
// block (experts_gemm.h has the product itself):
//
//   ffn_up      g = x Wg^T and u = x Wu^T together; act(g) u, rounded once to bf16, and what the backward pass needs
//   ffn_rows    y = h Wd^T; grad_x = [dg du] [Wg; Wu]
//   ffn_dh      dh = grad_y Wd, and from it and the saved g and u: dg, du and h
//   ffn_wgrad   [dg du]^T x and grad_y^T h
//
// Bound by the matrix pipes with hundreds of rows an expert, by the weights' bytes below.  On the Mixtral-like batch
// (8 experts, 1024 rows each, 4096 x 14336) and on 32 experts of 7168 x 2048 with 1024 rows: up 1.15 and 1.20
// PFLOP/s, down 1.17 and 1.12, grad_x 1.14 and 1.17, dh 0.86 and 0.95, weight gradients 1.02 and 1.02; one large
// library product reaches 1.57 (k-contiguous operands) and 1.30-1.36 (one k-strided).  dh has the lowest rate: its
// epilogue also moves g, u, dg, du and h, 1.2 GB in bf16 on the Mixtral-like batch.  At the rate of a copy that is 0.18 of
// the 0.28 ms by which it is slower than the other products; the rest is not explained (waves wait 37 % of their cycles).
#include <math.h>

#include <type_traits>

#include "experts_gemm.h"

namespace ms {
namespace {

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
int64_t places(int64_t tiles, int across) { return ((tiles + 3) / 4 * 4 * across + 255) / 256 * 256; }

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

// ---- the kernels ----
// The accumulators go to memory through LDS, packed to bf16, so that whole rows of a tile are written (256 or 512
// contiguous bytes a row) rather than the 8 bytes a lane holds.  h, dg and du are rounded to bf16 there because they are
// operands of the next products, whose matrix instructions take bf16; y and the gradients because they are bf16 outputs.

// Largest magnitude over the 32 features that the four lanes of a row hold in a and b; infinity if any is not
// finite.  Features past the width (`past`) count as zero.
__device__ __forceinline__ float group_top(f32x4 a, f32x4 b, bool past_a, bool past_b)
{
    float top = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = past_a ? 0.0f : fabsf(a[i]), y = past_b ? 0.0f : fabsf(b[i]);
        top = fmaxf(top, fmaxf(x, y));
        bad |= !(x <= 3.40282347e38f) || !(y <= 3.40282347e38f);
    }
    if (bad) top = __uint_as_float(0x7f800000u);
    top = fmaxf(top, __shfl_xor(top, 16, kWave));
    return fmaxf(top, __shfl_xor(top, 32, kWave));
}

// Rows an expert has on average, up to which tiles of 64 rows with two blocks a CU are taken.  Forward and backward pass
// in such tiles against higher ones, us, for 32 experts of 2048 x 2048, 8 of 4096 x 4096 and 48 of 1160 x 520:
//   even routing          40 rows  642 / 666, 725 / 728, 172 / 174    56 rows  738 / 682, 734 / 749, 214 / 187
//   popular experts       40 rows  677 / 775, 718 / 763, 200 / 244    56 rows  692 / 807, 689 / 796, 211 / 258
// From 48 rows on some of evenly loaded experts have a second tile, but with popular experts (Zipf, 1.2) the low tiles
// still win at 64 (707 / 791, 690 / 821, 221 / 271).  The host knows the mean alone; 56 lies between.
constexpr int kSmallRows = 56;
constexpr int kCUs = 256;
constexpr int kUpFeatures = kTileFeatures / 2;  // of h: each of them takes a gate and an up feature

template <bool Small>
__global__ __launch_bounds__(kGemmThreads, Small ? 4 : 2) void ffn_up_kernel(ExpertShape S, const char* xe, const char* w,
                                                                 char* h, SavedActs saved, int tile_rows, int across,
                                                                           GridSpan span)
{
    __shared__ __align__(1024) char lds[Lds<Small>::kBytes];
    const Place at = place_of(span, across);
    int row0, nr;
    const int bad = *S.status, e = segment_tile(S.offset, S.E, tile_rows, 32, at.tile, &row0, &nr);
    if (bad || e < 0) return;
    const int c0 = at.across * kUpFeatures, H = S.H, I = S.I;
    const int valid = min(kUpFeatures, I - c0);
    KContiguous r, f;
    r.init(H, H);
    f.init(H, H);
    // F0 is the gate's rows, F1 the up projection's: a wave gets both of the same features
    f.slot(0, w + ((int64_t)e * 2 * I + c0) * H * 2, valid);
    f.slot(1, w + ((int64_t)e * 2 * I + I + c0) * H * 2, valid);
    const int lane = lane_id(), wf = wave_id() & 3, groups = (I + kGroup8 - 1) / kGroup8;
    with_rows<Small>(nr, [&](auto mf) {
        constexpr int MF = decltype(mf)::value;
        Acc<MF> acc;
        row_slots<MF>(r, xe + (int64_t)row0 * H * 2, H, nr);
        tile_product<Small, MF>(r, f, H, lds, acc);
        typedef Stage<kUpFeatures * 2> Wide;
        typedef Stage<kUpFeatures> Narrow;
        char* const second = lds + Lds<Small>::kRows * kUpFeatures * 2;
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int row = row_of<MF>(m) + (lane & 15);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = 32 * wf + 16 * i + 4 * (lane >> 4);
                f32x4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float slope;
                    v[j] = acc[m][i][j] * gate_sigmoid(acc[m][i][j], S.c0, S.c1, &slope) * acc[m][2 + i][j];
                }
                *(u32x2*)Wide::at(lds, row, 2 * c) = pack4(v);
                if (saved.data && !saved.scale) *(u32x2*)Wide::at(second, row, 2 * c) = pack4(acc[m][i]);
            }
            if (!saved.scale) continue;
            const int c = 32 * wf + 4 * (lane >> 4);
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const f32x4 a = acc[m][2 * which], b = acc[m][2 * which + 1];
                const float step = step8(group_top(a, b, c0 + c >= I, c0 + c + 16 >= I)), inv = 1.0f / step;
                char* const to = second + which * Lds<Small>::kRows * kUpFeatures;
                *(unsigned*)Narrow::at(to, row, c) = pack8x4(a[0], a[1], a[2], a[3], inv);
                *(unsigned*)Narrow::at(to, row, c + 16) = pack8x4(b[0], b[1], b[2], b[3], inv);
                if (row < nr && lane < 16 && c0 + 32 * wf < I)
                    ((unsigned short*)saved.scale)[((int64_t)(row0 + row) * 2 + which) * groups + c0 / 32 + wf] =
                        (unsigned short)(__float_as_uint(step) >> 16);
            }
        }
        __syncthreads();
        Wide::store<u32x4, MF>(lds, nr, 2 * valid, h + ((int64_t)row0 * I + c0) * 2, (int64_t)I * 2);
        if (!saved.data) return;
        char* const out = (char*)saved.data + ((int64_t)row0 * 2 * I + c0) * (saved.scale ? 1 : 2);
        if (saved.scale) {
            Narrow::store<u32x2, MF>(second, nr, valid, out, (int64_t)2 * I);
            Narrow::store<u32x2, MF>(second + Lds<Small>::kRows * kUpFeatures, nr, valid, out + I, (int64_t)2 * I);
            return;
        }
        Wide::store<u32x4, MF>(second, nr, 2 * valid, out, (int64_t)4 * I);
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *(u32x2*)Wide::at(lds, row_of<MF>(m) + (lane & 15), 2 * (32 * wf + 16 * i + 4 * (lane >> 4))) =
                    pack4(acc[m][2 + i]);
        __syncthreads();
        Wide::store<u32x4, MF>(lds, nr, 2 * valid, out + (int64_t)2 * I, (int64_t)4 * I);
    });
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

// out[row] = in[row] F^T for the rows of every expert; in [P, K], out [P, N], F of an expert [N][K] (or, Strided,
// [K][N]) at w.
template <bool Strided, bool Small>
__global__ __launch_bounds__(kGemmThreads, Small ? 4 : 2) void ffn_rows_kernel(ExpertShape S, const char* in, int K,
                                                                   const char* w, int N, char* out,
                                                                              int tile_rows, int across, GridSpan span)
{
    __shared__ __align__(1024) char lds[Lds<Small>::kBytes];
    const Place at = place_of(span, across);
    int row0, nr;
    const int bad = *S.status, e = segment_tile(S.offset, S.E, tile_rows, 32, at.tile, &row0, &nr);
    if (bad || e < 0) return;
    const int n0 = at.across * kTileFeatures;
    KContiguous r;
    r.init(K, K);
    typename std::conditional<Strided, KStrided, KContiguous>::type f;
    f.init(Strided ? N : K, K);
    for (int i = 0; i < 2; ++i) {
        const int n = n0 + 128 * i;
        f.slot(i, w + (Strided ? (int64_t)e * K * N + n : ((int64_t)e * N + n) * K) * 2, N - n);
    }
    with_rows<Small>(nr, [&](auto mf) {
        constexpr int MF = decltype(mf)::value;
        Acc<MF> acc;
        row_slots<MF>(r, in + (int64_t)row0 * K * 2, K, nr);
        tile_product<Small, MF>(r, f, K, lds, acc);
        write_tile<MF>(lds, nr, min(N - n0, kTileFeatures), out + ((int64_t)row0 * N + n0) * 2, (int64_t)N * 2,
                       [&](int m, int n) { return pack4(acc[m][n]); });
    });
}

// Fragment rows [M0, M0 + MC) of dh, a slot's, with the saved pre-activations to dg, du and h.
template <bool Small, int M0, int MC, int MF>
__device__ __forceinline__ void dh_rows(const ExpertShape& S, char* lds, const Acc<MF>& acc, const SavedActs& saved,
                                        int row0, int nr, int n0, int valid, char* h, char* dgu)
{
    constexpr int kHalf = (Small ? 64 : 128) * kTileFeatures * 2, kFirst = M0 ? 32 * low_rows(MF) : 0;
    const int lane = lane_id(), I = S.I, groups = (I + kGroup8 - 1) / kGroup8;
    struct Held {
        u32x2 g, u;
        unsigned sg, su;
    };
    // rows and features outside the tile read their nearest neighbours: their results go nowhere
    const auto fetch = [&](int i, Held (&to)[4]) {
        const int64_t row = row0 + min(row_of<MF>(M0 + i) + (lane & 15), nr - 1);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int c = min(n0 + feature_of(n) + 4 * (lane >> 4), I - 4);
            const char* const from = (const char*)saved.data + (row * 2 * I + c) * (saved.scale ? 1 : 2);
            if (saved.scale) {
                to[n].g[0] = *(const unsigned*)from;
                to[n].u[0] = *(const unsigned*)(from + I);
                const unsigned short* const sc = (const unsigned short*)saved.scale + row * 2 * groups + c / kGroup8;
                to[n].sg = sc[0];
                to[n].su = sc[groups];
            } else {
                to[n].g = *(const u32x2*)from;
                to[n].u = *(const u32x2*)(from + 2 * I);
            }
        }
    };
    Held held[2][4];
    u32x2 hv[MC][4];
    fetch(0, held[0]);
#pragma unroll
    for (int i = 0; i < MC; ++i) {
        if (i + 1 < MC) fetch(i + 1, held[(i + 1) & 1]);
        const int row = row_of<MF>(M0 + i) - kFirst + (lane & 15);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const Held& q = held[i & 1][n];
            f32x4 g, u, vg, vu, vh;
            if (saved.scale) {
                const float sg = __uint_as_float(q.sg << 16), su = __uint_as_float(q.su << 16);
#pragma unroll
                for (int j = 0; j < 4; ++j) { g[j] = int8_of(q.g[0], j) * sg; u[j] = int8_of(q.u[0], j) * su; }
            } else {
                g = f32x4{bf16_lo(q.g[0]), bf16_hi(q.g[0]), bf16_lo(q.g[1]), bf16_hi(q.g[1])};
                u = f32x4{bf16_lo(q.u[0]), bf16_hi(q.u[0]), bf16_lo(q.u[1]), bf16_hi(q.u[1])};
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float slope;
                const float d = acc[M0 + i][n][j], s = gate_sigmoid(g[j], S.c0, S.c1, &slope), a = g[j] * s;
                vh[j] = a * u[j];
                vu[j] = d * a;
                vg[j] = d * (u[j] * fmaf(a * (1.0f - s), slope, s));  // a closed gate's 0 meets u first: d u may overflow
            }
            const int c = feature_of(n) + 4 * (lane >> 4);
            *(u32x2*)WideStage::at(lds, row, 2 * c) = pack4(vg);
            *(u32x2*)WideStage::at(lds + kHalf, row, 2 * c) = pack4(vu);
            hv[i][n] = pack4(vh);
        }
    }
    __syncthreads();
    const int64_t first = row0 + kFirst;
    char* const out = dgu + (first * 2 * I + n0) * 2;
    WideStage::store<u32x4, MC>(lds, nr - kFirst, 2 * valid, out, (int64_t)I * 4);
    WideStage::store<u32x4, MC>(lds + kHalf, nr - kFirst, 2 * valid, out + 2 * I, (int64_t)I * 4);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MC; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n)
            *(u32x2*)WideStage::at(lds, row_of<MF>(M0 + i) - kFirst + (lane & 15), 2 * (feature_of(n) + 4 * (lane >> 4))) =
                hv[i][n];
    __syncthreads();
    WideStage::store<u32x4, MC>(lds, nr - kFirst, 2 * valid, h + (first * I + n0) * 2, (int64_t)I * 2);
    __syncthreads();
}

template <bool Small>
__global__ __launch_bounds__(kGemmThreads, Small ? 4 : 2) void ffn_dh_kernel(ExpertShape S, const char* gy, const char* w,
                                                                 SavedActs saved, char* h, char* dgu, int tile_rows,
                                                                            int across, GridSpan span)
{
    __shared__ __align__(1024) char lds[Lds<Small>::kBytes];
    const Place at = place_of(span, across);
    int row0, nr;
    const int bad = *S.status, e = segment_tile(S.offset, S.E, tile_rows, 32, at.tile, &row0, &nr);
    if (bad || e < 0) return;
    const int n0 = at.across * kTileFeatures, H = S.H, I = S.I;
    KContiguous r;
    KStrided f;
    r.init(H, H);
    f.init(I, H);
    for (int i = 0; i < 2; ++i) f.slot(i, w + ((int64_t)e * H * I + n0 + 128 * i) * 2, I - n0 - 128 * i);
    const int valid = min(I - n0, kTileFeatures);
    with_rows<Small>(nr, [&](auto mf) {
        constexpr int MF = decltype(mf)::value;
        Acc<MF> acc;
        row_slots<MF>(r, gy + (int64_t)row0 * H * 2, H, nr);
        tile_product<Small, MF>(r, f, H, lds, acc);
        // a slot's rows at a time: dg and du go through LDS side by side, then h
        constexpr int A = low_rows(MF);
        dh_rows<Small, 0, A>(S, lds, acc, saved, row0, nr, n0, valid, h, dgu);
        if constexpr (MF > A) dh_rows<Small, A, MF - A>(S, lds, acc, saved, row0, nr, n0, valid, h, dgu);
    });
}

// out[e] = a^T b over the rows of expert e: both operands' k is the row.
__global__ __launch_bounds__(kGemmThreads, 2) void ffn_wgrad_kernel(ExpertShape S, const char* a, int na,
                                                                    const char* b, int nb, char* out, int down,
                                                                    int across, GridSpan span)
{
    __shared__ __align__(1024) char lds[Lds<false>::kBytes];
    if (*S.status) return;
    const Place at = place_of(span, across);
    const int e = at.tile / down, m0 = (at.tile - e * down) * kTileRows, n0 = at.across * kTileFeatures;
    if (e >= S.E) return;
    const int q0 = S.offset[e], rows = S.offset[e + 1] - q0;
    KStrided r, f;
    r.init(na, rows);
    f.init(nb, rows);
    for (int i = 0; i < 2; ++i) {
        r.slot(i, a + ((int64_t)q0 * na + m0 + 128 * i) * 2, na - m0 - 128 * i);
        f.slot(i, b + ((int64_t)q0 * nb + n0 + 128 * i) * 2, nb - n0 - 128 * i);
    }
    Acc<8> acc;
    tile_product<false, 8>(r, f, rows, lds, acc);
    write_tile<8>(lds, min(na - m0, kTileRows), min(nb - n0, kTileFeatures),
                  out + (((int64_t)e * na + m0) * nb + n0) * 2, (int64_t)nb * 2,
                  [&](int m, int n) { return pack4(acc[m][n]); });
}

int tiles_of(int n, int tile) { return (n + tile - 1) / tile; }

// The rows of a tile, 128 to 256, for an estimate of the time of `across` feature tiles: a tile takes 1.5 + its
// fragment rows (32 rows each), and the CUs take the tiles in rounds of 256, so that a few tiles more than whole rounds
// cost a round.  The rows of an expert are not known here; five counts around the mean stand for them, spread as
// even routing spreads them.  (8 experts of 1024 rows, 28672 to 4096: 1663 us with 192 rows against 1894 with 256;
// 16 experts of 375 rows, 2048 to 1000: 67 us with 160 against 85.  The estimates are 0.83 and 0.73 of the other.)
int pick_tile_rows(const ExpertShape& S, int across)
{
    const int used = S.P < S.E ? S.P : S.E;
    const double mean = (double)S.P / (used > 0 ? used : 1), spread = 0.6 * sqrt(mean);
    int best = kTileRows;
    double least = 0;
    for (int rows = kTileRows; rows >= 128; rows -= 32) {
        double tiles = 0, cost = 0;
        for (int j = -2; j <= 2; ++j) {
            const int64_t count = (int64_t)(mean + j * spread + 0.5), n = (count + rows - 1) / rows;
            tiles += (double)n;
            cost += n ? n * (1.5 + (double)((count + 32 * n - 1) / (32 * n))) : 0;
        }
        if (tiles == 0) continue;
        const double time = ceil(tiles / 5 * used * across / kCUs) * (cost / tiles);
        if (best == kTileRows && rows == kTileRows) least = time;
        if (time < 0.98 * least) {
            least = time;
            best = rows;
        }
    }
    return best;
}

// Calls launch(small, tile rows, blocks' grid, span) for a product of row tiles by `across` feature tiles.
template <class F>
hipError_t by_rows(const ExpertShape& S, int across, F&& launch)
{
    const auto with = [&](auto small) {
        constexpr bool kSmall = decltype(small)::value;
        const int rows = kSmall ? Lds<true>::kRows : pick_tile_rows(S, across);
        const int64_t tiles = (int64_t)S.P / rows + (S.P < S.E ? S.P : S.E);
        return launch_spans(places(tiles, across), kGemmThreads,
                            [&](dim3 grid, GridSpan span) { launch(small, rows, grid, span); });
    };
    return S.P <= (int64_t)kSmallRows * (S.P < S.E ? S.P : S.E) ? with(std::true_type()) : with(std::false_type());
}

}  // namespace

hipError_t launch_ffn_up(const ExpertShape& S, const void* xe, const void* w_gate_up, void* h, SavedActs saved,
                         hipStream_t s)
{
    const int across = tiles_of(S.I, kUpFeatures);
    return by_rows(S, across, [&](auto small, int rows, dim3 grid, GridSpan span) {
        ffn_up_kernel<decltype(small)::value><<<grid, kGemmThreads, 0, s>>>(
            S, (const char*)xe, (const char*)w_gate_up, (char*)h, saved, rows, across, span);
    });
}

hipError_t launch_ffn_down(const ExpertShape& S, const void* h, const void* w_down, void* ye, hipStream_t s)
{
    const int across = tiles_of(S.H, kTileFeatures);
    return by_rows(S, across, [&](auto small, int rows, dim3 grid, GridSpan span) {
        ffn_rows_kernel<false, decltype(small)::value><<<grid, kGemmThreads, 0, s>>>(
            S, (const char*)h, S.I, (const char*)w_down, S.H, (char*)ye, rows, across, span);
    });
}

hipError_t launch_ffn_dh(const ExpertShape& S, const void* grad_ye, const void* w_down, SavedActs saved, void* h,
                         void* dgu, hipStream_t s)
{
    const int across = tiles_of(S.I, kTileFeatures);
    return by_rows(S, across, [&](auto small, int rows, dim3 grid, GridSpan span) {
        ffn_dh_kernel<decltype(small)::value><<<grid, kGemmThreads, 0, s>>>(
            S, (const char*)grad_ye, (const char*)w_down, saved, (char*)h, (char*)dgu, rows, across, span);
    });
}

hipError_t launch_ffn_dx(const ExpertShape& S, const void* dgu, const void* w_gate_up, void* grad_xe, hipStream_t s)
{
    const int across = tiles_of(S.H, kTileFeatures);
    return by_rows(S, across, [&](auto small, int rows, dim3 grid, GridSpan span) {
        ffn_rows_kernel<true, decltype(small)::value><<<grid, kGemmThreads, 0, s>>>(
            S, (const char*)dgu, 2 * S.I, (const char*)w_gate_up, S.H, (char*)grad_xe, rows, across, span);
    });
}

hipError_t launch_ffn_wgrad(const ExpertShape& S, const void* a, int na, const void* b, int nb, void* out,
                            hipStream_t s)
{
    const int down = tiles_of(na, kTileRows), across = tiles_of(nb, kTileFeatures);
    return launch_spans(places((int64_t)S.E * down, across), kGemmThreads, [&](dim3 grid, GridSpan span) {
        ffn_wgrad_kernel<<<grid, kGemmThreads, 0, s>>>(S, (const char*)a, na, (const char*)b, nb, (char*)out, down,
                                                       across, span);
    });
}

}  // namespace ms
