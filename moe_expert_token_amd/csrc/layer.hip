// layer.hip -- a whole mixture-of-experts layer for a few tokens in three kernels: the router's scores, the two
// projections, the down projection with the weighted sum.  Very few scores are made in the projections: two kernels.
//
// The weights of the chosen experts are the cost (experts_stream.h has how a wave streams them); all else is latency.
// So nothing goes through memory that a block can find out by itself: every block of the projections chooses the
// experts of all tokens anew from the scores and makes its own list of row tiles, where a plan, a dispatch and a copy of
// the rows would be three launches.
//
//   scores   l = x w^T, one expert a block: products of bf16 numbers are exact in fp32, and are summed in 64 bits, in
//            the order that layer.h sets for all calls
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

__device__ __forceinline__ double as_double(unsigned bits) { return (double)__uint_as_float(bits); }

// Experts [Experts blockIdx.x, ...) and Tokens tokens a block; its waves share H.  What a number costs is its way
// to 64 bits, so with many tokens four experts share it (48 tokens, 256 experts, H = 7168: 17 us).
template <int Tokens, int Experts, int Threads>
__global__ __launch_bounds__(Threads) void layer_scores_kernel(LayerShape S, Rule rule, const u32x4* x,
                                                                     const u32x4* w, int columns)
{
    constexpr int kSums = Tokens * Experts;
    static_assert(Threads == kSumParts * kWave, "a wave is a part of the sums");
    __shared__ double part[kSumParts][kSums];
    const int e0 = blockIdx.x * Experts, t0 = blockIdx.y * Tokens, V = S.H / 8;
    if (e0 == 0 && t0 == 0)
        for (int i = threadIdx.x; i < columns; i += Threads) S.arrived[i] = 0;
    double sum[kSums] = {};  // [Experts][Tokens]
#pragma unroll 1
    for (int v = threadIdx.x; v < V; v += Threads) {
        u32x4 a[Experts], b[Tokens];  // tokens and experts past the last repeat it
#pragma unroll
        for (int i = 0; i < Experts; ++i) a[i] = w[(int64_t)min(e0 + i, S.E - 1) * V + v];
#pragma unroll
        for (int t = 0; t < Tokens; ++t) b[t] = x[(int64_t)min(t0 + t, S.T - 1) * V + v];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                double wd[Experts];
#pragma unroll
                for (int i = 0; i < Experts; ++i) wd[i] = as_double(h ? a[i][c] & 0xffff0000u : a[i][c] << 16);
#pragma unroll
                for (int t = 0; t < Tokens; ++t) {
                    const double xd = as_double(h ? b[t][c] & 0xffff0000u : b[t][c] << 16);
#pragma unroll
                    for (int i = 0; i < Experts; ++i) sum[i * Tokens + t] = fma(wd[i], xd, sum[i * Tokens + t]);
                }
            }
    }
    double mine;
    const int which = wave_sums(sum, &mine);
    if ((lane_id() & (kWave / kSums - 1)) == 0) part[wave_id()][which] = mine;
    __syncthreads();
    const int t = t0 + (int)threadIdx.x % Tokens, e = e0 + (int)threadIdx.x / Tokens;
    if ((int)threadIdx.x >= kSums || t >= S.T || e >= S.E) return;
    const double l = parts_total([&](int i) { return part[i][threadIdx.x]; });
    const int64_t at = (int64_t)t * S.E + e;
    S.logit[at] = (float)l;
    S.key[at] = ordered_key(rule.bias ? score64(l) + (double)rule.bias[e] : l);
}

template <int Tokens, int Experts, int Threads>
hipError_t launch_scores(const LayerShape& S, const Rule& rule, const LayerCall& C, hipStream_t s)
{
    const dim3 grid((S.E + Experts - 1) / Experts, (S.T + Tokens - 1) / Tokens);
    layer_scores_kernel<Tokens, Experts, Threads><<<grid, Threads, 0, s>>>(S, rule, (const u32x4*)C.x,
                                                                           (const u32x4*)C.w_router, (S.H + 63) / 64);
    return hipGetLastError();
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

// Where there is a wave for each token and expert, and their sums are short, a block of the projections makes the scores
// itself: one launch less.  Us a call in a graph, with and without (bf16 experts half as wide): one token, 8 experts, H = 128
// 11.9 / 13.4, 512 13.4 / 15.0, 1024 16.4 / 17.5, 2048 22.7 / 23.1, 4096 37.0 / 35.9; four tokens, 8 experts, H = 1024 20.7 /
// 18.7, 4096 83 / 70; one token, 64 experts, H = 512 18.1 / 15.1.
constexpr int kOwnPairs = kWaves;
constexpr int64_t kOwnProducts = 1 << 15;

bool own_scores(const LayerShape& S)
{
    const int64_t pairs = (int64_t)S.T * S.E;
    return pairs <= kOwnPairs && pairs * S.H <= kOwnProducts;
}

// What every block of the projections finds out for itself.
struct Choice {
    unsigned long long tokens[kMaxExperts];
    int first[kMaxExperts];
    int tile[kLayerPairs];
    int wave_sum[kWaves];
    int tiles;
    unsigned long long key[kOwnPairs];  // of all tokens and experts, where there are few
    float logit[kOwnPairs];
};

__device__ __forceinline__ void own_scores_of(const LayerShape& S, const Rule& rule, const u32x4* x, const u32x4* w,
                                              Choice& C)
{
    const int V = S.H / 8;
    for (int p = wave_id(); p < S.T * S.E; p += kWaves) {
        const int t = p / S.E, e = p - t * S.E;
        double sum[kSumParts] = {};
        for (int v0 = lane_id(); v0 < V; v0 += kSumParts * kWave) {
#pragma unroll
            for (int i = 0; i < kSumParts; ++i) {
                const int v = v0 + i * kWave;
                if (v >= V) break;
                const u32x4 a = w[(int64_t)e * V + v], b = x[(int64_t)t * V + v];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    sum[i] = fma(as_double(a[c] << 16), as_double(b[c] << 16), sum[i]);
                    sum[i] = fma(as_double(a[c] & 0xffff0000u), as_double(b[c] & 0xffff0000u), sum[i]);
                }
            }
        }
        double l;
        if (V <= kWave) {  // the other parts are 0
            double first[1] = {sum[0]};
            wave_sums(first, &l);
        } else {
            double mine;
            wave_sums(sum, &mine);  // part i in lanes 8 i on
            l = parts_total([&](int i) { return lane_value(mine, i * (kWave / kSumParts)); });
        }
        if (lane_id() == 0) {
            C.logit[p] = (float)l;
            C.key[p] = ordered_key(rule.bias ? score64(l) + (double)rule.bias[e] : l);
        }
    }
}

// Sorts two keys with their experts, the larger first; of equal ones the one that comes first stays first.
__device__ __forceinline__ void order(unsigned long long& a, unsigned long long& b, int& ea, int& eb)
{
    const bool swap = b > a || (b == a && eb < ea);
    const unsigned long long k = swap ? b : a;
    const int e = swap ? eb : ea;
    b = swap ? a : b;
    eb = swap ? ea : eb;
    a = k;
    ea = e;
}

// The k largest of the E keys of N tokens, by one wave with Each keys of a token a lane: the tokens' bits in the experts'
// words, and lane j's expert of slot j.  A choice is a chain of some twenty dependent steps, so two tokens go side by side.
template <int Each, int N>
__device__ __forceinline__ void choose_tokens(const LayerShape& S, bool own, const int (&t)[N], Choice& C,
                                              int (&chosen)[N])
{
    const int lane = lane_id();
    unsigned long long key[N][Each];
    int expert[N][Each];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < Each; ++i) {
            const int e = lane + i * kWave;
            expert[n][i] = e;
            if (Each == 1 && own) key[n][i] = C.key[t[n] * S.E + min(e, S.E - 1)];
            else key[n][i] = S.key[(int64_t)t[n] * S.E + min(e, S.E - 1)];
            if (e >= S.E) key[n][i] = 0;
        }
    if constexpr (Each == 4) {  // a lane's keys in order, so that only the first is looked at
#pragma unroll
        for (int n = 0; n < N; ++n) {
            order(key[n][0], key[n][1], expert[n][0], expert[n][1]);
            order(key[n][2], key[n][3], expert[n][2], expert[n][3]);
            order(key[n][0], key[n][2], expert[n][0], expert[n][2]);
            order(key[n][1], key[n][3], expert[n][1], expert[n][3]);
            order(key[n][1], key[n][2], expert[n][1], expert[n][2]);
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) chosen[n] = 0;
#pragma unroll 1
    for (int j = 0; j < S.k; ++j) {
        unsigned long long best[N], tie[N];
        unsigned top[N];
        int at[N], e[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            best[n] = key[n][0];
            at[n] = expert[n][0];
            if constexpr (Each > 4) {
#pragma unroll
                for (int i = 1; i < Each; ++i)
                    if (key[n][i] > best[n]) { best[n] = key[n][i]; at[n] = expert[n][i]; }
            }
            top[n] = wave_max((unsigned)(best[n] >> 32));
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            tie[n] = __ballot((unsigned)(best[n] >> 32) == top[n]);
            e[n] = __builtin_amdgcn_readlane(at[n], __builtin_ctzll(tie[n]));
            if (tie[n] & (tie[n] - 1)) e[n] = wave_argmax(best[n], at[n]);
            if (lane == j) chosen[n] = e[n];
            if constexpr (Each > 4) {
#pragma unroll
                for (int i = 0; i < Each; ++i)
                    if (expert[n][i] == e[n]) key[n][i] = 0;
            } else {
                const bool pop = at[n] == e[n];
#pragma unroll
                for (int i = 0; i < Each; ++i) {
                    const int from = i + 1 < Each ? i + 1 : i;
                    key[n][i] = pop ? (i + 1 < Each ? key[n][from] : 0) : key[n][i];
                    expert[n][i] = pop ? (i + 1 < Each ? expert[n][from] : -1) : expert[n][i];
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
        if (lane < S.k) atomicOr(&C.tokens[chosen[n]], 1ull << t[n]);
}

// The gates of a token, for the kernel that follows and for the user: lane j's of slot j.
__device__ __forceinline__ void write_gates(const LayerShape& S, const Rule& rule, const float* l, int t, int chosen,
                                            int32_t* topk_idx, float* topk_w)
{
    const int lane = lane_id(), E = S.E, k = S.k;
    float most = -__builtin_inff(), all = 0;
    if (!rule.sigmoid) {
        for (int e = lane; e < E; e += kWave) most = fmaxf(most, l[e]);
        most = wave_max(most);
        if (!rule.normalize) {
            for (int e = lane; e < E; e += kWave) all += expf(l[e] - most);
            all = wave_total(all);
        }
    }
    const float w = gate_of(rule, k, l[chosen], most, all);
    if (lane < k) {
        S.gate[t * k + lane] = w;
        if (topk_idx) topk_idx[t * k + lane] = chosen;
        if (topk_w) topk_w[t * k + lane] = w;
    }
}

// Rows of an expert's tile p of `rows`: the first and how many.
__device__ __forceinline__ int tile_rows(unsigned long long tokens, int rows, int p)
{
    return min(rows, (int)__popcll(tokens) - p * rows);
}

// Chooses the experts of all tokens and lists the tiles of up to `rows` rows.  What the kernel that follows needs of it is
// written down once: by block t for token t, by the first block for all.  (A block more that does nothing else is a
// round more where the others fill the card: 37.5 us against 31.8, one token, 256 4-bit experts of 7168 x 2048.)
__device__ __forceinline__ void choose(const LayerShape& S, const Rule& rule, int rows, const char* x, const char* w,
                                       Choice& C, int32_t* topk_idx, float* topk_w)
{
    const int lane = lane_id(), wave = wave_id(), E = S.E, k = S.k;
    const bool own = w != nullptr;
    for (int e = threadIdx.x; e < E; e += kThreads) C.tokens[e] = 0;
    if (own) {
        own_scores_of(S, rule, (const u32x4*)x, (const u32x4*)w, C);
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < (S.H + 63) / 64; i += kThreads) S.arrived[i] = 0;
    }
    __syncthreads();
    const auto some = [&](auto each) {
        constexpr int Each = decltype(each)::value, N = Each > 4 ? 1 : 2;
#pragma unroll 1
        for (int t0 = wave; t0 < S.T; t0 += N * kWaves) {
            int chosen[N], t[N];
            if (N == 1 || t0 + kWaves >= S.T) {
                int one[1] = {t0}, its[1];
                choose_tokens<Each, 1>(S, own, one, C, its);
                t[0] = t0;
                chosen[0] = its[0];
                if (N > 1) t[N - 1] = -1;
            } else {
#pragma unroll
                for (int n = 0; n < N; ++n) t[n] = t0 + n * kWaves;
                choose_tokens<Each, N>(S, own, t, C, chosen);
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (t[n] < 0 || t[n] % (int)gridDim.x != (int)blockIdx.x) continue;
                if (own) write_gates(S, rule, C.logit + t[n] * E, t[n], chosen[n], topk_idx, topk_w);
                else write_gates(S, rule, S.logit + (int64_t)t[n] * E, t[n], chosen[n], topk_idx, topk_w);
                if (lane < k) S.row_of[t[n] * k + lane] = chosen[n];  // its row, once the first rows are known
            }
        }
    };
    if (E <= 64) some(std::integral_constant<int, 1>());
    else if (E <= 256) some(std::integral_constant<int, 4>());
    else some(std::integral_constant<int, 16>());
    __syncthreads();
    // rows and tiles before each expert, two experts a thread, counted together: 512 at most of each
    int count[2], sum = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * threadIdx.x + i, n = e < E ? __popcll(C.tokens[e]) : 0;
        count[i] = n | (n + rows - 1) / rows << 16;
        sum += count[i];
    }
    const int upto = wave_scan(sum);
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
    for (int t = blockIdx.x; t < S.T; t += gridDim.x)
        for (int j = threadIdx.x; j < k; j += kThreads) {
            const int e = S.row_of[t * k + j];
            S.row_of[t * k + j] = C.first[e] + __popcll(C.tokens[e] & ((1ull << t) - 1));
        }
    if (blockIdx.x) return;
    for (int i = threadIdx.x; i < C.tiles; i += kThreads) {
        const int e = C.tile[i] & 0xffff, p = C.tile[i] >> 16;
        S.tile[i] = make_int4(e, C.first[e] + p * rows, tile_rows(C.tokens[e], rows, p), 0);
    }
    if (threadIdx.x == 0) *S.tiles = C.tiles;
}

struct Weights {
    const char *w, *scale;
    int across;  // blocks over the features
};

template <int Group, int Rows, int Ways, bool Whole, bool Staged>
__global__ __launch_bounds__(kThreads, Rows == 16 ? 4 : 2) void layer_up_kernel(LayerShape S, Rule rule, const char* x, const char* w,
                                                            Weights A, int32_t* topk_idx, float* topk_w)
{
    typedef LayerSplit<Rows, Ways> P;
    constexpr int kOut = 32;  // output features of a wave
    __shared__ __align__(16) char lds[Staged ? P::kStage : P::kSums];
    __shared__ Choice C;
    choose(S, rule, Rows, x, w, C, topk_idx, topk_w);
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

// y goes to memory and comes from there, not from an L2 that is one of eight (sc1, agent scope): so a block's y is there
// for every other one as soon as its stores are done, which a wait for them shows.  Fences would do the same by writing
// back and dropping the whole L2, for each tile (890 us against 311 without any, 48 tokens, 256 experts of 2048 to 7168).
constexpr int kAgent = 16;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const float* y, int64_t bytes)
{
    const uint64_t a = (uint64_t)y;
    const uint64_t p = (unsigned)__builtin_amdgcn_readfirstlane((int)a) |
                       (uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)(a >> 32)) << 32;
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, __builtin_amdgcn_readfirstlane((int)(unsigned)bytes),
                                             0x00020000);
}

// Columns [n0, n0 + width) of out: the rows' y, weighted and added in the order of the slots.
__device__ __forceinline__ void combine(const LayerShape& S, const int* row_of, const float* gate, const void* residual,
                                        void* out, int n0, int width)
{
    const int quads = (min(width, S.H - n0) + 3) / 4;
    const __amdgpu_buffer_rsrc_t rows = rows_of(S.y, (int64_t)S.P * S.H * 4);
    for (int i = threadIdx.x; i < S.T * quads; i += kThreads) {
        const int t = i / quads, n = n0 + 4 * (i - t * quads);
        const int64_t at = (int64_t)t * S.H + n;
        u32x2 r = {0, 0};
        if (residual) r = *(const u32x2*)((const unsigned short*)residual + at);
        f32x4 sum = {0, 0, 0, 0};
#pragma unroll 8
        for (int j = 0; j < S.k; ++j) {
            const float w = gate[t * S.k + j];
            const unsigned from = ((unsigned)row_of[t * S.k + j] * S.H + n) * 4;
            const f32x4 y = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, from, 0, kAgent));
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[c] = fmaf(w, y[c], sum[c]);
        }
        if (residual) {
            sum[0] += bf16_lo(r[0]);
            sum[1] += bf16_hi(r[0]);
            sum[2] += bf16_lo(r[1]);
            sum[3] += bf16_hi(r[1]);
        }
        *(u32x2*)((unsigned short*)out + at) = u32x2{bf16_pack2(sum[0], sum[1]), bf16_pack2(sum[2], sum[3])};
    }
}

template <int Group, int Rows, int Ways, bool Whole, bool Staged>
__global__ __launch_bounds__(kThreads, Rows == 16 ? 4 : 2) void layer_down_kernel(LayerShape S, Weights A, const void* residual, void* out)
{
    typedef LayerSplit<Rows, Ways> P;
    constexpr int kOut = 64;
    __shared__ __align__(16) char lds[Staged ? P::kStage : P::kSums];
    __shared__ int last, row_of[kLayerPairs];
    __shared__ float gate[kLayerPairs];
    for (int p = threadIdx.x; p < S.P; p += kThreads) {  // a barrier comes before they are read
        row_of[p] = S.row_of[p];
        gate[p] = S.gate[p];
    }
    const int ks = wave_id() % P::KS, fs = wave_id() / P::KS, K = S.I, N = S.H;
    const int tiles = *S.tiles, items = tiles * A.across;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int tile = item / A.across, place = item - tile * A.across;
        const int4 what = S.tile[tile];
        const int e = __builtin_amdgcn_readfirstlane(what.x), nr = __builtin_amdgcn_readfirstlane(what.z);
        const int64_t row0 = __builtin_amdgcn_readfirstlane(what.y);
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
            const __amdgpu_buffer_rsrc_t rows = rows_of(S.y + row0 * N, (int64_t)nr * N * 4);
            for (int i = ks * kWave + lane_id(); i < nr * kOut; i += P::KS * kWave) {
                const int r = i / kOut, f = i % kOut, n = n0 + f;
                const float v = total(f >> 4, r, f);
                if (n < N) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rows, (r * N + n) * 4, 0, kAgent);
            }
        };
        if (Rows == 16 || nr <= 16) run(std::integral_constant<int, 1>());
        else run(std::integral_constant<int, 2>());
        // every wave's y is in memory before the block's arrival; the last to arrive finds them all there
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0)
            last = __hip_atomic_fetch_add(S.arrived + place, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == tiles - 1;
        __syncthreads();
        if (last) combine(S, row_of, gate, residual, out, place * P::FS * kOut, P::FS * kOut);
    }
}

constexpr int kResident = 512;  // two blocks a CU

template <int Group, int Rows, int Ways, bool Whole, bool Staged>
hipError_t launch_up(const LayerShape& S, const Rule& rule, const LayerCall& C, hipStream_t s)
{
    constexpr int kOut = 32 * LayerSplit<Rows, Ways>::FS;
    const Weights A{(const char*)C.up, (const char*)C.up_scale, (S.I + kOut - 1) / kOut};
    const int64_t items = (int64_t)((S.P < S.E ? S.P : S.E) + S.P / Rows) * A.across;
    const int grid = (int)(items < kResident ? items : kResident);
    layer_up_kernel<Group, Rows, Ways, Whole, Staged><<<grid, kThreads, 0, s>>>(
        S, rule, (const char*)C.x, own_scores(S) ? (const char*)C.w_router : nullptr, A, C.topk_idx, C.topk_w);
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

// A block's eight waves are the ways of a sum of bf16 weights, whatever its length.  They are dealt chunks of 128 k four at
// a time, so a short sum keeps some of them only: one wave of eight with k up to 512, two up to 1024, four up to 2048; all
// from 4096 on.  Us a call with eight ways and with two, which are dealt alike: one token, 64 experts of 2048 x 1024 28.0 /
// 58.6, 16 tokens 161 / 177, 64 tokens 184 / 200; one token, 8 of 7168 x 2048 144.7 / 143.7.  Of 4-bit weights, dealt chunk
// by chunk, two ways share a sum where k is short, unless that leaves half of the card without work: groups of 128, one
// token, 8 experts of 1024 x 512 15.2 / 19.8, 64 experts of 7168 x 2048 54.4 / 53.0, 256 of them 53.2 / 50.9, 16 tokens, 64
// of them 310 / 299, 64 tokens, 64 of 2048 x 1024 82.1 / 75.1; groups of 64 15.3 / 19.9, 56.3 / 55.3, 54.2 / 51.4, 312 / 305,
// 83.1 / 74.6; groups of 32 15.6 / 20.9, 59.1 / 59.1, 57.4 / 55.6, 332 / 321, 84.8 / 77.5.  (There, as it is, the projections
// of 7168 k have eight, and the down projection two.)  The scales of the features have to fit LDS, or come from memory.
constexpr int kFewItems = 128;

template <int Group, int Rows, bool Up>
hipError_t launch_one(const LayerShape& S, const Rule& rule, const LayerCall& C, hipStream_t s)
{
    const int K = Up ? S.H : S.I;
#define MS_LAYER(WAYS, WHOLE, STAGED) \
    (Up ? launch_up<Group, Rows, WAYS, WHOLE, STAGED>(S, rule, C, s) : launch_down<Group, Rows, WAYS, WHOLE, STAGED>(S, rule, C, s))
    if constexpr (Group == 0) {
        return K % kChunk ? MS_LAYER(8, false, false) : MS_LAYER(8, true, false);
    } else {
        const int N = Up ? S.I : S.H, wide = (Up ? 32 : 64) * LayerSplit<Rows, 2>::FS;
        const bool few = K < kLongK && (int64_t)(S.P < S.E ? S.P : S.E) * ((N + wide - 1) / wide) >= kFewItems;
        const auto fits = [&](int ways) { return (int64_t)64 * (kWaves / ways) * (K / Group) * 2 <= 64 << 10; };
        const bool two = fits(2) && few;
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

// Rows an expert has on average, up to which tiles have 16 of them: two blocks fit a CU then, but an expert with more
// has its weights read again.  Us a call with 16 and with 32, for 64 experts of 2048 x 1024, 8 of 4096 x 4096 (where the
// rule loses 5 % in bf16) and 16 of 2048 x 2048: bf16, 4 rows 172 / 179, 184 / 175, 92 / 94; 10 rows -, 194 / 183, 103 / 105;
// 12 rows -, 218 / 187, 118 / 106; groups of 128, 4 rows 62 / 73, 55 / 65, 44 / 45; 10 rows -, 65 / 76, 58 / 59; 12 rows -, 80 /
// 82, 72 / 65.
constexpr int kRowsOf16 = 10;

template <int Group>
hipError_t launch_rows(const LayerShape& S, const Rule& rule, const LayerCall& C, hipStream_t s)
{
    return S.P <= (int64_t)kRowsOf16 * (S.P < S.E ? S.P : S.E) ? launch_both<Group, 16>(S, rule, C, s)
                                                               : launch_both<Group, 32>(S, rule, C, s);
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
    S->tile = (int4*)take(P * 16);
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
    const hipError_t e = own_scores(S) ? hipSuccess
                         : S.T == 1 ? launch_scores<1, 1, 512>(S, rule, C, s)
                         : S.T <= 4 ? launch_scores<4, 1, 512>(S, rule, C, s)
                                    : launch_scores<8, 4, 512>(S, rule, C, s);
    if (e != hipSuccess) return e;
    switch (C.group) {
        case 32: return launch_rows<32>(S, rule, C, s);
        case 64: return launch_rows<64>(S, rule, C, s);
        case 128: return launch_rows<128>(S, rule, C, s);
        default: return launch_rows<0>(S, rule, C, s);
    }
}

}  // namespace ms
