// layer.hip -- a whole mixture-of-experts layer for a few tokens in three kernels: the router's scores, the two
// projections, the down projection with the weighted sum.
//
// The weights of the chosen experts are the cost (experts_stream.h has how a wave streams them); all else is latency.
// So nothing goes through memory that a block can find out by itself: every block of the projections chooses the
// experts of all tokens anew from the scores (2 us, beside weights of 25 to 600) and makes its own list of row tiles,
// where a plan, a dispatch and a copy of the rows would be three launches.
//
//   scores   l = x w^T, one expert a block: products of bf16 numbers are exact in fp32, and are summed in 64 bits, so
//            that the choice does not depend on the sum's order
//   up       the choice, the list of tiles (an expert and up to 16 or 32 of its tokens), act(g) u for each, fp32
//            rounded once to bf16.  The tokens of an expert are the bits of one 64-bit word.
//   down     y = h Wd^T in fp32 for each tile; the block that finishes a column last (a counter a column, cleared by
//            `scores`) has all experts' y of it, and adds them up in the order of the slots: no atomics on values, the
//            same bits whichever block that is
#include <math.h>

#include "experts_stream.h"
#include "layer.h"

namespace ms {
namespace {

using namespace stream;

constexpr int kScoreThreads = 256;
constexpr int kScoreTokens = 8;  // of a block

__device__ __forceinline__ double as_double(unsigned bits) { return (double)__uint_as_float(bits); }

// One expert a block, up to eight tokens; the four waves share H.
__global__ __launch_bounds__(kScoreThreads) void layer_scores_kernel(LayerShape S, Rule rule, const u32x4* x,
                                                                     const u32x4* w, int columns)
{
    __shared__ double part[kScoreThreads / kWave][kScoreTokens];
    const int e = blockIdx.x, t0 = blockIdx.y * kScoreTokens, n = min(kScoreTokens, S.T - t0), V = S.H / 8;
    if (e == 0 && t0 == 0)
        for (int i = threadIdx.x; i < columns; i += kScoreThreads) S.arrived[i] = 0;
    double sum[kScoreTokens] = {};
    for (int v = threadIdx.x; v < V; v += kScoreThreads) {
        const u32x4 a = w[(int64_t)e * V + v];
        double wd[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            wd[2 * c] = as_double(a[c] << 16);
            wd[2 * c + 1] = as_double(a[c] & 0xffff0000u);
        }
#pragma unroll
        for (int t = 0; t < kScoreTokens; ++t) {
            if (t >= n) break;
            const u32x4 b = x[(int64_t)(t0 + t) * V + v];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sum[t] = fma(wd[2 * c], as_double(b[c] << 16), sum[t]);
                sum[t] = fma(wd[2 * c + 1], as_double(b[c] & 0xffff0000u), sum[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kScoreTokens; ++t) {
        if (t >= n) break;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) sum[t] += __shfl_xor(sum[t], d, kWave);
        if (lane_id() == 0) part[wave_id()][t] = sum[t];
    }
    __syncthreads();
    if ((int)threadIdx.x >= n) return;
    const int t = threadIdx.x;
    const double l = (part[0][t] + part[1][t]) + (part[2][t] + part[3][t]);
    const int64_t at = (int64_t)(t0 + t) * S.E + e;
    S.logit[at] = (float)l;
    S.key[at] = ordered_key(rule.bias ? score64(l) + (double)rule.bias[e] : l);
}

// How a block's eight waves share its work, as stream::Split, for tiles of Rows rows.
template <int Rows, int Ways>
struct LayerSplit {
    static constexpr int kRows = Rows;
    static constexpr int KS = Ways;
    static constexpr int FS = kWaves / KS;
    static constexpr int kSums = kWaves * kGroupsOf16 * (kRows / 16) * kWave * 16;
    static constexpr int kStage = 64 << 10;  // room for scales, then sums
    static_assert(kStage >= kSums, "sums fit");
};

constexpr int kMaxExperts = 1024;

// What every block of the projections finds out for itself.
struct Choice {
    unsigned long long tokens[kMaxExperts];
    int first[kMaxExperts];
    int tile[kLayerPairs];
    int wave_sum[kWaves];
    int tiles;
};

// Chooses the experts of all tokens and lists the tiles of up to `rows` rows.  The keys of a wave's token are kept in
// `keys` (E of them a wave).  The first block writes the choice down for the kernel that follows and for the user.
__device__ __forceinline__ void choose(const LayerShape& S, const Rule& rule, int rows, unsigned long long* keys,
                                       Choice& C, int32_t* topk_idx, float* topk_w)
{
    const int lane = lane_id(), wave = wave_id(), E = S.E, k = S.k;
    const bool write = blockIdx.x == 0;
    for (int e = threadIdx.x; e < E; e += kThreads) C.tokens[e] = 0;
    __syncthreads();
    unsigned long long* const mine = keys + wave * E;
    for (int t = wave; t < S.T; t += kWaves) {
        for (int e = lane; e < E; e += kWave) mine[e] = S.key[(int64_t)t * E + e];
        float most = -__builtin_inff(), all = 0;
        if (!rule.sigmoid && write) {
            for (int e = lane; e < E; e += kWave) most = fmaxf(most, S.logit[(int64_t)t * E + e]);
            most = wave_max(most);
            if (!rule.normalize) {
                for (int e = lane; e < E; e += kWave) all += expf(S.logit[(int64_t)t * E + e] - most);
                all = wave_total(all);
            }
        }
        int chosen = 0;  // lane j's: slot j's expert
        for (int j = 0; j < k; ++j) {
            unsigned long long best = 0;
            int at = E;
            for (int e = lane; e < E; e += kWave)
                if (mine[e] > best) { best = mine[e]; at = e; }
            const int e = wave_argmax(best, at);
            if (lane == j) chosen = e;
            if (lane == (e & (kWave - 1))) mine[e] = 0;
            if (lane == 0) atomicOr(&C.tokens[e], 1ull << t);
        }
        if (write) {
            const float w = gate_of(rule, k, S.logit[(int64_t)t * E + chosen], most, all);
            if (lane < k) {
                S.gate[t * k + lane] = w;
                if (topk_idx) topk_idx[t * k + lane] = chosen;
                if (topk_w) topk_w[t * k + lane] = w;
                S.row_of[t * k + lane] = chosen;  // its row, once the first rows are known
            }
        }
    }
    __syncthreads();
    // rows and tiles before each expert, two experts a thread, counted together: 512 at most of each
    int count[2], sum = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * threadIdx.x + i, n = e < E ? __popcll(C.tokens[e]) : 0;
        count[i] = n | (n + rows - 1) / rows << 16;
        sum += count[i];
    }
    const int upto = wave_inclusive_scan(sum);
    if (lane == kWave - 1) C.wave_sum[wave] = upto;
    __syncthreads();
    int before = upto - sum, total = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        if (i < wave) before += C.wave_sum[i];
        total += C.wave_sum[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * threadIdx.x + i;
        if (e < E) C.first[e] = before & 0xffff;
        for (int p = 0; p < count[i] >> 16; ++p) C.tile[(before >> 16) + p] = e | p << 16;
        before += count[i];
    }
    if (threadIdx.x == 0) C.tiles = total >> 16;
    __syncthreads();
    if (!write) return;
    for (int e = threadIdx.x; e < E; e += kThreads) {
        S.tokens[e] = C.tokens[e];
        S.first[e] = C.first[e];
    }
    for (int i = threadIdx.x; i < C.tiles; i += kThreads) S.tile[i] = C.tile[i];
    if (threadIdx.x == 0) *S.tiles = C.tiles;
    for (int p = threadIdx.x; p < S.P; p += kThreads) {
        const int e = S.row_of[p], t = p / k;
        S.row_of[p] = C.first[e] + __popcll(C.tokens[e] & ((1ull << t) - 1));
    }
}

struct Weights {
    const char *w, *scale;
    int across;  // blocks over the features
};

// Rows of an expert's tile p of `rows`: the first and how many.
__device__ __forceinline__ int tile_rows(unsigned long long tokens, int rows, int p)
{
    return min(rows, (int)__popcll(tokens) - p * rows);
}

template <int Group, int Rows, int Ways, bool Whole, bool Staged>
__global__ __launch_bounds__(kThreads) void layer_up_kernel(LayerShape S, Rule rule, const char* x, Weights A,
                                                            int32_t* topk_idx, float* topk_w)
{
    typedef LayerSplit<Rows, Ways> P;
    constexpr int kOut = 32;  // output features of a wave
    __shared__ __align__(16) char lds[P::kStage];
    __shared__ Choice C;
    choose(S, rule, Rows, (unsigned long long*)lds, C, topk_idx, topk_w);
    const int ks = wave_id() % P::KS, fs = wave_id() / P::KS, K = S.H, N = S.I;
    const int items = C.tiles * A.across;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int tile = item / A.across, place = item - tile * A.across;
        const int e = __builtin_amdgcn_readfirstlane(C.tile[tile] & 0xffff);
        const int p = __builtin_amdgcn_readfirstlane(C.tile[tile] >> 16);
        const unsigned long long tokens = C.tokens[e];
        const int nr = __builtin_amdgcn_readfirstlane(tile_rows(tokens, Rows, p));
        Source<Group, true> from;
        from.init(K);
        from.x.init(x, (int64_t)S.T * K * 2);
        {  // the tokens of this lane's rows
            unsigned long long m = tokens;
            for (int i = 0; i < p * Rows; ++i) m &= m - 1;
            const int r = lane_id() & 15;
            from.picked[0] = from.picked[1] = kOutside;
            for (int i = 0; i < nr; ++i, m &= m - 1) {
                const unsigned at = (unsigned)__builtin_ctzll(m) * from.xld;
                if (r == i) from.picked[0] = at;
                if (r + 16 == i) from.picked[1] = at;
            }
        }
        const int n0 = (place * P::FS + fs) * kOut;  // this wave's first output feature
        const int64_t wrow = (int64_t)e * 2 * N + n0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t first = wrow + (i ? N : 0);
            from.side(i, A.w + first * from.ld, A.scale + first * from.sld, N - n0);
        }
        if constexpr (Staged) stage_scales<P>(lds, from, ks, fs);
        const int64_t row0 = C.first[e] + p * Rows;
        const auto run = [&](auto tiles) {
            const auto total = sum_up<Group, P, decltype(tiles)::value, Whole, Staged>(lds, from, ks, fs);
            for (int i = ks * kWave + lane_id(); i < nr * kOut; i += P::KS * kWave) {
                const int r = i / kOut, f = i % kOut, n = n0 + f;
                float slope;
                const float g = total(f >> 4, r, f), u = total(2 + (f >> 4), r, f);
                if (n < N)
                    ((unsigned short*)S.h)[(row0 + r) * N + n] = bf16_of(g * gate_sigmoid(g, S.c0, S.c1, &slope) * u);
            }
        };
        if (Rows == 16 || nr <= 16) run(std::integral_constant<int, 1>());
        else run(std::integral_constant<int, 2>());
        __syncthreads();  // the sums' room is the next tile's
    }
}

// Columns [n0, n0 + width) of out: the rows' y, weighted and added in the order of the slots.
__device__ __forceinline__ void combine(const LayerShape& S, const void* residual, void* out, int n0, int width)
{
    const int quads = (min(width, S.H - n0) + 3) / 4;
    for (int i = threadIdx.x; i < S.T * quads; i += kThreads) {
        const int t = i / quads, n = n0 + 4 * (i - t * quads);
        f32x4 sum = {0, 0, 0, 0};
        for (int j = 0; j < S.k; ++j) {
            const float w = S.gate[t * S.k + j];
            const f32x4 y = *(const f32x4*)(S.y + (int64_t)S.row_of[t * S.k + j] * S.H + n);
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[c] = fmaf(w, y[c], sum[c]);
        }
        const int64_t at = (int64_t)t * S.H + n;
        if (residual) {
            const u32x2 r = *(const u32x2*)((const unsigned short*)residual + at);
            sum[0] += bf16_lo(r[0]);
            sum[1] += bf16_hi(r[0]);
            sum[2] += bf16_lo(r[1]);
            sum[3] += bf16_hi(r[1]);
        }
        *(u32x2*)((unsigned short*)out + at) = u32x2{bf16_pack2(sum[0], sum[1]), bf16_pack2(sum[2], sum[3])};
    }
}

template <int Group, int Rows, int Ways, bool Whole, bool Staged>
__global__ __launch_bounds__(kThreads) void layer_down_kernel(LayerShape S, Weights A, const void* residual, void* out)
{
    typedef LayerSplit<Rows, Ways> P;
    constexpr int kOut = 64;
    __shared__ __align__(16) char lds[Staged ? P::kStage : P::kSums];
    __shared__ int last;
    const int ks = wave_id() % P::KS, fs = wave_id() / P::KS, K = S.I, N = S.H;
    const int tiles = *S.tiles, items = tiles * A.across;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int tile = item / A.across, place = item - tile * A.across;
        const int what = S.tile[tile], e = what & 0xffff, p = what >> 16;
        const int nr = __builtin_amdgcn_readfirstlane(tile_rows(S.tokens[e], Rows, p));
        const int64_t row0 = S.first[e] + p * Rows;
        Source<Group> from;
        from.init(K);
        from.x.init(S.h + row0 * K * 2, (int64_t)nr * K * 2);
        const int n0 = (place * P::FS + fs) * kOut;
        const int64_t wrow = (int64_t)e * N + n0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t first = wrow + 32 * i;
            from.side(i, A.w + first * from.ld, A.scale + first * from.sld, N - n0 - 32 * i);
        }
        if constexpr (Staged) stage_scales<P>(lds, from, ks, fs);
        const auto run = [&](auto tiles) {
            const auto total = sum_up<Group, P, decltype(tiles)::value, Whole, Staged>(lds, from, ks, fs);
            for (int i = ks * kWave + lane_id(); i < nr * kOut; i += P::KS * kWave) {
                const int r = i / kOut, f = i % kOut, n = n0 + f;
                const float v = total(f >> 4, r, f);
                if (n < N) S.y[(row0 + r) * N + n] = v;
            }
        };
        if (Rows == 16 || nr <= 16) run(std::integral_constant<int, 1>());
        else run(std::integral_constant<int, 2>());
        // this block's y before its arrival; the last to arrive sees them all
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) last = atomicAdd(S.arrived + place, 1) == tiles - 1;
        __syncthreads();
        if (last) {
            __threadfence();
            combine(S, residual, out, place * P::FS * kOut, P::FS * kOut);
        }
    }
}

constexpr int kResident = 512;  // two blocks a CU

template <int Group, int Rows, int Ways, bool Whole, bool Staged>
hipError_t launch_up(const LayerShape& S, const Rule& rule, const LayerCall& C, hipStream_t s)
{
    constexpr int kOut = 32 * LayerSplit<Rows, Ways>::FS;
    const Weights A{(const char*)C.up, (const char*)C.up_scale, (S.I + kOut - 1) / kOut};
    const int64_t items = (int64_t)((S.P < S.E ? S.P : S.E) + S.P / Rows) * A.across;
    layer_up_kernel<Group, Rows, Ways, Whole, Staged><<<(int)(items < kResident ? items : kResident), kThreads, 0, s>>>(
        S, rule, (const char*)C.x, A, C.topk_idx, C.topk_w);
    return hipGetLastError();
}

template <int Group, int Rows, int Ways, bool Whole, bool Staged>
hipError_t launch_down(const LayerShape& S, const Rule&, const LayerCall& C, hipStream_t s)
{
    constexpr int kOut = 64 * LayerSplit<Rows, Ways>::FS;
    const Weights A{(const char*)C.down, (const char*)C.down_scale, (S.H + kOut - 1) / kOut};
    const int64_t items = (int64_t)((S.P < S.E ? S.P : S.E) + S.P / Rows) * A.across;
    layer_down_kernel<Group, Rows, Ways, Whole, Staged><<<(int)(items < kResident ? items : kResident), kThreads, 0, s>>>(
        S, A, C.residual, C.out);
    return hipGetLastError();
}

// The rules of experts_few.hip: few ways over k where k is short, room for the scales permitting.
template <int Group, int Rows, bool Up>
hipError_t launch_one(const LayerShape& S, const Rule& rule, const LayerCall& C, hipStream_t s)
{
    const int K = Up ? S.H : S.I;
#define MS_LAYER(WAYS, WHOLE, STAGED) \
    (Up ? launch_up<Group, Rows, WAYS, WHOLE, STAGED>(S, rule, C, s) : launch_down<Group, Rows, WAYS, WHOLE, STAGED>(S, rule, C, s))
    if constexpr (Group == 0) {
        if (K % kChunk) return MS_LAYER(8, false, false);
        return K >= kLongK ? MS_LAYER(8, true, false) : MS_LAYER(2, true, false);
    } else {
        const auto fits = [&](int ways) { return (int64_t)64 * (kWaves / ways) * (K / Group) * 2 <= 64 << 10; };
        const bool two = fits(2) && K < kLongK;
        if (!two && !fits(8)) return MS_LAYER(8, false, false);
        if constexpr (Group % kChunk != 0)  // K is a multiple of the group
            if (K % kChunk) return two ? MS_LAYER(2, false, true) : MS_LAYER(8, false, true);
        return two ? MS_LAYER(2, true, true) : MS_LAYER(8, true, true);
    }
#undef MS_LAYER
}

template <int Group, int Rows>
hipError_t launch_both(const LayerShape& S, const Rule& rule, const LayerCall& C, hipStream_t s)
{
    const hipError_t e = launch_one<Group, Rows, true>(S, rule, C, s);
    return e != hipSuccess ? e : launch_one<Group, Rows, false>(S, rule, C, s);
}

template <int Group>
hipError_t launch_rows(const LayerShape& S, const Rule& rule, const LayerCall& C, hipStream_t s)
{
    // up to 16 tokens no expert has more rows
    return S.T <= 16 ? launch_both<Group, 16>(S, rule, C, s) : launch_both<Group, 32>(S, rule, C, s);
}

}  // namespace

size_t layer_workspace(LayerShape* S, char* base)
{
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        char* const p = base + at;
        at = (at + bytes + 255) & ~(size_t)255;
        return p;
    };
    const size_t T = S->T, E = S->E, P = S->P;
    S->key = (unsigned long long*)take(T * E * 8);
    S->logit = (float*)take(T * E * 4);
    S->tokens = (unsigned long long*)take(E * 8);
    S->first = (int*)take(E * 4);
    S->tile = (int*)take(P * 4);
    S->tiles = (int*)take(4);
    S->row_of = (int*)take(P * 4);
    S->gate = (float*)take(P * 4);
    S->arrived = (int*)take(((size_t)S->H + 63) / 64 * 4);
    S->h = take(P * S->I * 2);
    S->y = (float*)take(P * S->H * 4);
    return at;
}

hipError_t launch_layer(const LayerShape& S, const Rule& rule, const LayerCall& C, hipStream_t s)
{
    layer_scores_kernel<<<dim3(S.E, (S.T + kScoreTokens - 1) / kScoreTokens), kScoreThreads, 0, s>>>(
        S, rule, (const u32x4*)C.x, (const u32x4*)C.w_router, (S.H + 63) / 64);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    switch (C.group) {
        case 32: return launch_rows<32>(S, rule, C, s);
        case 64: return launch_rows<64>(S, rule, C, s);
        case 128: return launch_rows<128>(S, rule, C, s);
        default: return launch_rows<0>(S, rule, C, s);
    }
}

}  // namespace ms
