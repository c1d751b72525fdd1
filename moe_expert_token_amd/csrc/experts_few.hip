// experts_few.hip -- the experts' block where an expert has few rows: the
// weights' bytes are the cost, so every wave streams weights from memory
// straight into registers (experts_stream.h).  Weights are bf16, or 4-bit with
// group scales.
//
// Kernel times: four tokens that hit 5 bf16 experts of 4096 x 14336, 197 + 140
// us (1.76 GB, 5.2 TB/s); 4-bit weights in groups of 128, 256 experts of 7168 x
// 2048, one token 25 + 16 us (182 MB of weights, 4.4 TB/s); 48 tokens 633 + 311
// us (4.7 GB, 5.0 TB/s), the matrix pipes 16 % busy, waves waiting for data 45 %
// of their cycles.  With 203 tokens on 8 experts of 4096 x 14336, groups of 32,
// weights are read about once (0.58 and 0.36 GB) and the memory is not the
// limit: two waves a SIMD wait 47 % of their cycles for an instruction to issue
// and 27 % for data.
#include "experts_stream.h"

namespace ms {
namespace {

using namespace stream;

struct FewArgs {
    const char* x;         // [P][K] bf16
    const char* w;         // [E][rows of both sides][K]
    const char* scale;
    char* out;             // [P][N] bf16
    int K, N;              // N: features of the output
    SavedActs saved;       // of the projections
    int across;            // blocks over N
};

// Keeps a row's pre-activation of feature n, the gate's (side 0) or the up projection's; 32 neighbouring lanes hold
// a group of an 8-bit checkpoint (zeros past the row's end).
__device__ __forceinline__ void save(const SavedActs& to, int64_t row, int side, int n, int N, float v, bool ok)
{
    const int64_t at = row * 2 * N + (side ? N : 0) + n;
    if (!to.scale) {
        if (ok) ((unsigned short*)to.data)[at] = bf16_of(v);
        return;
    }
    float top = ok ? fabsf(v) : 0.0f;
    if (!(top <= 3.40282347e38f)) top = __uint_as_float(0x7f800000u);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    const float step = step8(top);
    if (ok) ((unsigned char*)to.data)[at] = (unsigned char)pack8x4(v, v, v, v, 1.0f / step);
    if (ok && n % kGroup8 == 0)
        ((unsigned short*)to.scale)[(row * 2 + side) * ((N + kGroup8 - 1) / kGroup8) + n / kGroup8] =
            (unsigned short)(__float_as_uint(step) >> 16);
}

// Up: features c and c + N of the weights make feature c of the output, h = act(gate) * up.
template <int Group, bool Up, bool Few, int Ways, bool Whole, bool Staged>
__global__ __launch_bounds__(kThreads) void ffn_few_kernel(ExpertShape S, FewArgs A, GridSpan span)
{
    typedef Split<Group, Few, Ways> P;
    constexpr int kOut = Up ? 32 : 64;  // output features of a wave
    __shared__ __align__(16) char lds[Staged ? P::kStage : P::kSums];
    const int b = span_block(span), tile = b / A.across, place = b - tile * A.across;
    int row0, nr;
    const int bad = *S.status, e = segment_tile(S.offset, S.E, P::kRows, 16, tile, &row0, &nr);
    if (bad || e < 0) return;
    const int ks = wave_id() % P::KS, fs = wave_id() / P::KS, K = A.K, N = A.N;
    Source<Group> from;
    from.init(K);
    from.x.init(A.x + (int64_t)row0 * K * 2, (int64_t)nr * K * 2);
    const int n0 = (place * P::FS + fs) * kOut;  // this wave's first output feature
    const int64_t wrow = (int64_t)e * (Up ? 2 * N : N) + n0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t first = wrow + (Up ? (i ? N : 0) : 32 * i);
        from.side(i, A.w + first * from.ld, A.scale + first * from.sld, Up ? N - n0 : N - n0 - 32 * i);
    }
    if constexpr (Staged) stage_scales<P>(lds, from, ks, fs);
    const auto run = [&](auto tiles) {
        constexpr int RT = decltype(tiles)::value;
        const auto total = sum_up<Group, P, RT, Whole, Staged>(lds, from, ks, fs);
        // whole rows a turn, so that the lanes of a group stay together
        for (int i = ks * kWave + lane_id(); i < (nr * kOut + kWave - 1) / kWave * kWave; i += P::KS * kWave) {
            const int r = i / kOut, f = i % kOut, n = n0 + f;
            const bool ok = r < nr && n < N;
            const int64_t row = row0 + r;
            if constexpr (!Up) {
                const float v = total(f >> 4, min(r, nr - 1), f);
                if (ok) ((unsigned short*)A.out)[row * N + n] = bf16_of(v);
            } else {
                float slope;
                const float g = total(f >> 4, min(r, nr - 1), f), u = total(2 + (f >> 4), min(r, nr - 1), f);
                if (ok) ((unsigned short*)A.out)[row * N + n] = bf16_of(g * gate_sigmoid(g, S.c0, S.c1, &slope) * u);
                if (Group == 0 && A.saved.data) {
                    save(A.saved, row, 0, n, N, g, ok);
                    save(A.saved, row, 1, n, N, u, ok);
                }
            }
        }
    };
    if constexpr (Few) {
        run(std::integral_constant<int, 1>());
    } else {
        if constexpr (P::kRows == 32) {
            if (nr <= 16) run(std::integral_constant<int, 1>());
            else run(std::integral_constant<int, 2>());
        } else {
            if (nr <= 32) run(std::integral_constant<int, 2>());
            else run(std::integral_constant<int, 4>());
        }
    }
}

template <int Group, bool Up, bool Few, int Ways, bool Whole, bool Staged>
hipError_t launch(const ExpertShape& S, FewArgs A, hipStream_t s)
{
    typedef Split<Group, Few, Ways> P;
    const int out = (Up ? 32 : 64) * P::FS;
    A.across = (A.N + out - 1) / out;
    const int64_t tiles = (int64_t)S.P / P::kRows + (S.P < S.E ? S.P : S.E);
    return launch_spans(tiles * A.across, kThreads, [&](dim3 grid, GridSpan span) {
        ffn_few_kernel<Group, Up, Few, Ways, Whole, Staged><<<grid, kThreads, 0, s>>>(S, A, span);
    });
}

// Rows an expert has on average, of those that can have one.
bool few_each(const ExpertShape& S, int rows) { return S.P <= (int64_t)rows * (S.P < S.E ? S.P : S.E); }

template <int Group, bool Up, bool Few, int Ways>
hipError_t launch_w4_ways(const ExpertShape& S, const FewArgs& A, hipStream_t s)
{
    if constexpr (Group % kChunk != 0)  // K is a multiple of the group
        if (A.K % kChunk) return launch<Group, Up, Few, Ways, false, true>(S, A, s);
    return launch<Group, Up, Few, Ways, true, true>(S, A, s);
}

// Few ways over k leave more features to a block, which then share its rows' loads; many ways fit longer rows of
// scales, and keep every wave busy where there is little else to do (203 tokens, 14336 to 4096, groups of 32: 153 us
// with eight ways against 446 with two and scales from memory; 4096 to 2 x 14336: 313 with two, 346 with eight).
template <int Group, bool Up, bool Few>
hipError_t launch_w4_rows(const ExpertShape& S, const FewArgs& A, hipStream_t s)
{
    if (scales_fit<Group, Few, 2>(A.K) && (!Few || A.K < kLongK)) return launch_w4_ways<Group, Up, Few, 2>(S, A, s);
    if (scales_fit<Group, Few, 8>(A.K)) return launch_w4_ways<Group, Up, Few, 8>(S, A, s);
    return launch<Group, Up, Few, 8, false, false>(S, A, s);
}

template <int Group, bool Up>
hipError_t launch_w4_group(const ExpertShape& S, const FewArgs& A, hipStream_t s)
{
    // Tiles of 16 rows against higher ones, us, groups of 128, for 32 experts of 2048 x 2048, 8 of 4096 x 4096 and 64 of
    // 1024 x 2048: 8 rows on average 52 / 53, 50 / 63, 55 / 60; 12 rows 77 / 62, 54 / 69, 76 / 69; 16 rows 88 / 69, 75 / 82,
    // 85 / 76.  More experts, more of them with a second tile of 16: 12 lies between.
    return few_each(S, 12) ? launch_w4_rows<Group, Up, true>(S, A, s) : launch_w4_rows<Group, Up, false>(S, A, s);
}

template <bool Up>
hipError_t launch_w4(const ExpertShape& S, const FewArgs& A, int group, hipStream_t s)
{
    if (group == 128) return launch_w4_group<128, Up>(S, A, s);
    return group == 64 ? launch_w4_group<64, Up>(S, A, s) : launch_w4_group<32, Up>(S, A, s);
}

template <bool Up>
hipError_t launch_bf16(const ExpertShape& S, const FewArgs& A, hipStream_t s)
{
    if (A.K % kChunk) return launch<0, Up, true, 8, false, false>(S, A, s);
    return A.K >= kLongK ? launch<0, Up, true, 8, true, false>(S, A, s) : launch<0, Up, true, 2, true, false>(S, A, s);
}

}  // namespace

// The streams against the tiles of experts_ffn, us, for 32 experts of 2048 x 2048, 8 of 4096 x 4096 and 64 of 1024 x
// 2048: 8 rows on average 173 / 200, 171 / 203, 160 / 159; 10 rows 174 / 199, 172 / 203, 203 / 160; 12 rows 227 / 200,
// 173 / 203, 206 / 161; 16 rows 216 / 199, 209 / 203, 214 / 162.  The host knows the mean alone: all of 80 tokens on one
// of 8 experts of 4096 x 4096 take 101 us in streams, which read its weights five times, and 75 in tiles.
bool ffn_is_few(const ExpertShape& S) { return few_each(S, 10); }

hipError_t launch_few_up(const ExpertShape& S, const void* xe, const void* w_gate_up, void* h, SavedActs saved,
                         hipStream_t s)
{
    return launch_bf16<true>(S, FewArgs{(const char*)xe, (const char*)w_gate_up, nullptr, (char*)h, S.H, S.I, saved, 0}, s);
}

hipError_t launch_few_down(const ExpertShape& S, const void* h, const void* w_down, void* ye, hipStream_t s)
{
    return launch_bf16<false>(S, FewArgs{(const char*)h, (const char*)w_down, nullptr, (char*)ye, S.I, S.H, SavedActs{}, 0}, s);
}

hipError_t launch_w4_up(const ExpertShape& S, const void* xe, const void* q, const void* scale, int group, void* h,
                        hipStream_t s)
{
    return launch_w4<true>(S, FewArgs{(const char*)xe, (const char*)q, (const char*)scale, (char*)h, S.H, S.I, SavedActs{}, 0}, group, s);
}

hipError_t launch_w4_down(const ExpertShape& S, const void* h, const void* q, const void* scale, int group, void* ye,
                          hipStream_t s)
{
    return launch_w4<false>(S, FewArgs{(const char*)h, (const char*)q, (const char*)scale, (char*)ye, S.I, S.H, SavedActs{}, 0}, group, s);
}

}  // namespace ms
