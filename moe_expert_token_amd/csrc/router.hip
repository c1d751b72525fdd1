// router.hip -- the router of many rows and its backward pass.
//
//   logits   x W^T by the tile product of experts_gemm.h, a tile of 64 rows and 256 experts a block, H split over
//            blocks where there are few tiles (partial sums in fp32 in the workspace)
//   choose   a wave a row: the partial sums' sum, the k largest keys, the gates
//   dlogits  a wave a row: the gates' gradients to the logits', bf16
//   grad_x   dl W by tiles, grad_x_in added in fp32 before the one rounding
//   grad_w   dl^T x by tiles, T split over blocks, and the sum of their parts
//
// The choice has to be that of exact sums, and matrix instructions sum in fp32.  So `choose` knows how far a logit may
// be off: a sum of products computed in `steps` roundings one after another is off by at most steps 2^-23 sum |x w|, and
// sum |x w| <= ||x|| ||w||.  The norms come out of the same product for nothing (the fragments are in registers: one of
// four waves squares a tile of k).  Two neighbours among the k + 1 largest keys that are nearer than twice that bound
// are summed again, in 64 bits, by the wave that found them.
#include <math.h>

#include "experts_tiles.h"
#include "layer.h"

namespace ms {
namespace {

constexpr int kTokens = 64;  // rows of a logits tile

// How the logits' product is split: `splits` parts of `each` elements of H (a multiple of the tile's 64).
struct Cut {
    int splits, each, ld;  // ld: a row of partial sums, E rounded up to 4
    float gamma;           // a logit is off by at most gamma ||x|| ||w||
};

struct Partial {
    float *sum, *x2, *w2;  // [splits][T][ld], [splits][T] and [splits][E]: parts of logits and of squared norms
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float squares(bf16x8 v, float sum)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2 p = {v[2 * i], v[2 * i + 1]};
        sum = __builtin_amdgcn_fdot2_f32_bf16(p, p, sum, false);
    }
    return sum;
}

// Adds up the squares of rows and features; of the waves that share rows or features one does it for a tile of k.
template <int MF>
struct Squares {
    float row[MF], feature[4];

    template <int N>
    __device__ __forceinline__ void rows(int kt, int first, const bf16x8 (&r)[N][2])
    {
        if ((kt & 3) != (wave_id() & 3)) return;
#pragma unroll
        for (int i = 0; i < N; ++i) row[first + i] = squares(r[i][1], squares(r[i][0], row[first + i]));
    }
    __device__ __forceinline__ void features(int kt, const bf16x8 (&f0)[2][2], const bf16x8 (&f1)[2][2])
    {
        if ((kt & 1) != (wave_id() >> 2)) return;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            feature[i] = squares(f0[i][1], squares(f0[i][0], feature[i]));
            feature[2 + i] = squares(f1[i][1], squares(f1[i][0], feature[2 + i]));
        }
    }
};

// Sum over the four lanes that hold a row's (or feature's) k.
__device__ __forceinline__ float over_k(float v)
{
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
}

__global__ __launch_bounds__(kGemmThreads, 4) void router_logits_kernel(RouterShape S, Cut cut, Partial P, const char* x,
                                                                        const char* w, int tiles, GridSpan span)
{
    __shared__ __align__(1024) char lds[Lds<true>::kBytes];
    constexpr int MF = 2;
    // the parts of H vary fastest: with 1, 2, 4 or 8 of them an XCD's L2 holds one part of the weights, not all
    const int b = span_block(span), part = b % cut.splits, at = b / cut.splits, tile = at % tiles;
    const int t0 = tile * kTokens, e0 = at / tiles * kTileFeatures, k0 = part * cut.each;
    const int nr = min(kTokens, S.T - t0), K = min(cut.each, S.H - k0), lane = lane_id(), wave = wave_id();
    KContiguous r, f;
    r.init(S.H, K);
    f.init(S.H, K);
    row_slots<MF>(r, x + ((int64_t)t0 * S.H + k0) * 2, S.H, nr);
    for (int i = 0; i < 2; ++i) {
        const int e = e0 + 128 * i;
        f.slot(i, w + ((int64_t)e * S.H + k0) * 2, S.E - e);
    }
    Squares<MF> see = {};
    Acc<MF> acc;
    tile_product<true, MF>(r, f, K, lds, acc, see);
    float* const to = P.sum + ((int64_t)part * S.T + t0) * cut.ld + e0;
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int row = row_of<MF>(m) + (lane & 15), c = feature_of(n) + 4 * (lane >> 4);
            if (row < nr && e0 + c < cut.ld) *(f32x4*)(to + (int64_t)row * cut.ld + c) = acc[m][n];
        }
    // LDS is free: [4][64] parts of the rows' squares, then [2][256] of the features'
    float* const rows = (float*)lds;
    float* const features = rows + 4 * kTokens;
#pragma unroll
    for (int m = 0; m < MF; ++m) {
        const float v = over_k(see.row[m]);
        if (lane < 16) rows[(wave & 3) * kTokens + row_of<MF>(m) + lane] = v;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const float v = over_k(see.feature[n]);
        if (lane < 16) features[(wave >> 2) * kTileFeatures + feature_of(n) + lane] = v;
    }
    __syncthreads();
    const int i = threadIdx.x;
    if (i < nr && e0 == 0)
        P.x2[(int64_t)part * S.T + t0 + i] = (rows[i] + rows[kTokens + i]) + (rows[2 * kTokens + i] + rows[3 * kTokens + i]);
    if (tile == 0 && i < kTileFeatures && e0 + i < S.E) P.w2[part * S.E + e0 + i] = features[i] + features[kTileFeatures + i];
}

// ---- the choice ----

constexpr int kChooseWaves = 4;

// x . w[e] in 64 bits, the same in every lane.
__device__ __forceinline__ double exact_logit(const u32x4* x, const u32x4* w, int V)
{
    double sum = 0;
    for (int v = lane_id(); v < V; v += kWave) {
        const u32x4 a = x[v], b = w[v];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            sum = fma((double)bf16_lo(a[c]), (double)bf16_lo(b[c]), sum);
            sum = fma((double)bf16_hi(a[c]), (double)bf16_hi(b[c]), sum);
        }
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d, kWave);
    return sum;
}

// As ordered_key, of fp32 keys.
__device__ __forceinline__ unsigned ordered_key32(float v)
{
    if (v != v) v = -__builtin_inff();
    v += 0.0f;
    const unsigned u = __float_as_uint(v);
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(unsigned u) { return __uint_as_float(u >> 31 ? u & 0x7fffffffu : ~u); }

struct ChooseArgs {
    const u32x4 *x, *w;
    int32_t* idx;
    float *gate, *logits;
};

// All of a row's keys in 64 bits, and the k largest: where keys crowd, or norms say nothing.  With `zero` every logit is 0.
__device__ __forceinline__ int choose_exact(const RouterShape& S, const Rule& rule, bool zero, const u32x4* x,
                                            const u32x4* w, unsigned long long* keys)
{
    const int lane = lane_id(), V = S.H / 8;
#pragma unroll 1
    for (int e0 = 0; e0 < S.E; e0 += kWave) {
        double l = 0;  // lane i's: expert e0 + i
        if (!zero)
#pragma unroll 1
            for (int i = 0; i < kWave && e0 + i < S.E; ++i) {
                const double d = exact_logit(x, w + (int64_t)(e0 + i) * V, V);
                if (lane == i) l = d;
            }
        const int e = e0 + lane;
        if (e < S.E) keys[e] = ordered_key(rule.bias ? score64(l) + (double)rule.bias[e] : l);
    }
    int chosen = 0;
#pragma unroll 1
    for (int j = 0; j < S.k; ++j) {
        unsigned long long best = 0;
        int at = lane;
        for (int e = lane; e < S.E; e += kWave)
            if (keys[e] > best) { best = keys[e]; at = e; }
        const int e = wave_argmax(best, at);
        if (lane == j) chosen = e;
        if (lane == (e & (kWave - 1))) keys[e] = 0;
    }
    return chosen;
}

// A wave a row; Each logits a lane.
template <int Each>
__global__ __launch_bounds__(kChooseWaves * kWave) void router_choose_kernel(RouterShape S, Rule rule, Cut cut, Partial P,
                                                                             ChooseArgs A, GridSpan span)
{
    __shared__ unsigned long long keys[kChooseWaves][Each * kWave];
    const int lane = lane_id(), E = S.E, k = S.k, V = S.H / 8;
    const int64_t t = (int64_t)span_block(span) * kChooseWaves + wave_id();
    if (t >= S.T) return;
    float l[Each], w2 = 0;
    float x2 = 0;
    for (int s = 0; s < cut.splits; ++s) x2 += P.x2[(int64_t)s * S.T + t];
    const float* const sums = P.sum + t * cut.ld;
    const int64_t next = (int64_t)S.T * cut.ld;
#pragma unroll
    for (int i = 0; i < Each; ++i) {
        const int e = lane + i * kWave;
        l[i] = 0;
        float n = 0;
        if (e < E)
            for (int s = 0; s < cut.splits; ++s) {
                l[i] += sums[s * next + e];
                n += P.w2[s * E + e];
            }
        if (e < E && A.logits) A.logits[t * E + e] = l[i];
        w2 = n != n || n > w2 ? n : w2;  // a NaN stays
        if (w2 != w2) w2 = __builtin_inff();
    }
    w2 = wave_max(w2);
    // how far a key may be off.  Squares that underflow say nothing, unless all is zero
    const bool tiny = x2 < 8e-25f || w2 < 8e-25f;
    bool exact = !(x2 <= 1e38f && w2 <= 1e38f), zero = w2 == 0.0f;
    if (!exact && tiny && !zero) {
        unsigned any = 0;
        for (int v = lane; v < V; v += kWave) {
            const u32x4 a = A.x[t * V + v];
            any |= (a[0] | a[1] | a[2] | a[3]) & 0x7fff7fffu;
        }
        zero = __ballot(any != 0) == 0;
        exact = !zero;
    }
    float slack = zero ? 0.0f : cut.gamma * sqrtf(x2) * sqrtf(w2) * 1.01f;
    float bias[Each], most_bias = 0;
    if (rule.bias) {
#pragma unroll
        for (int i = 0; i < Each; ++i) {
            const int e = lane + i * kWave;
            bias[i] = e < E ? rule.bias[e] : 0.0f;
            if (fabsf(bias[i]) <= 3.4e38f) most_bias = fmaxf(most_bias, fabsf(bias[i]));
        }
        // a sigmoid's slope is a quarter at most; its own roundings and the sum's in fp32
        slack = 0.25f * slack + 4.8e-7f * (1.0f + wave_max(most_bias));
    }
    int chosen = 0;  // lane j's: the expert of slot j
    if (!exact) {
        unsigned key[Each];
#pragma unroll
        for (int i = 0; i < Each; ++i) {
            const int e = lane + i * kWave;
            key[i] = e < E ? ordered_key32(rule.bias ? 1.0f / (1.0f + expf(-l[i])) + bias[i] : l[i]) : 0;
        }
        // lane j's: the j-th largest key and its expert, k of them and those that may be as large as the k-th
        int mine = 0, m = 0;
        unsigned my_key = 0;
        float least = 0;
        for (;;) {
            unsigned best = key[0];
            int at = lane;
#pragma unroll
            for (int i = 1; i < Each; ++i)
                if (key[i] > best) { best = key[i]; at = lane + i * kWave; }
            const unsigned top = wave_max(best);
            if (top == 0) break;  // all experts are listed
            if (m >= k && (slack == 0 || !(key_value(top) >= least - 2 * slack))) break;
            if (m == kWave) { exact = true; break; }
            const unsigned long long tie = __ballot(best == top);
            const int e = (tie & (tie - 1)) == 0 ? __builtin_amdgcn_readlane(at, __builtin_ctzll(tie))
                                                 : (int)~wave_max(best == top ? ~(unsigned)at : 0u);
            if (lane == m) {
                mine = e;
                my_key = top;
            }
#pragma unroll
            for (int i = 0; i < Each; ++i)
                if (lane + i * kWave == e) key[i] = 0;
            if (++m == k) least = key_value(top);
        }
        if (!exact) {
            const float v = key_value(my_key);
            const float after = __shfl_down(v, 1, kWave);
            // the slack is 0 where all keys are exact: equal ones are listed in the order of their indexes
            const bool near = slack > 0 && lane + 1 < m && v - after <= 2 * slack;
            unsigned long long again = __ballot(near);
            again |= again << 1;
            if (again == 0) {
                chosen = mine;
            } else {
                double key64 = (double)v;
                for (unsigned long long left = again; left; left &= left - 1) {
                    const int i = __builtin_ctzll(left), e = __builtin_amdgcn_readlane(mine, i);
                    const double d = zero ? 0.0 : exact_logit(A.x + t * V, A.w + (int64_t)e * V, V);
                    const double kd = rule.bias ? score64(d) + (double)rule.bias[e] : d;
                    if (lane == i) key64 = kd;
                }
                const unsigned long long u = lane < m ? ordered_key(key64) : 0;
                int rank = 0;
                for (int i = 0; i < m; ++i) {
                    const unsigned long long o =
                        (unsigned long long)(unsigned)__builtin_amdgcn_readlane((int)(u >> 32), i) << 32 |
                        (unsigned)__builtin_amdgcn_readlane((int)(unsigned)u, i);
                    const int e = __builtin_amdgcn_readlane(mine, i);
                    rank += o > u || (o == u && e < mine);
                }
                // to the lane of its slot; lanes past the candidates rank behind them
                if (lane >= m) rank = lane;
                chosen = __builtin_amdgcn_ds_permute(rank * 4, mine);
            }
        }
    }
    if (exact) chosen = choose_exact(S, rule, zero, A.x + t * V, A.w, keys[wave_id()]);
    float most = -__builtin_inff(), all = 0;
    if (!rule.sigmoid) {
#pragma unroll
        for (int i = 0; i < Each; ++i)
            if (lane + i * kWave < E) most = fmaxf(most, l[i]);
        most = wave_max(most);
        if (!rule.normalize) {
#pragma unroll
            for (int i = 0; i < Each; ++i)
                if (lane + i * kWave < E) all += expf(l[i] - most);
            all = wave_total(all);
        }
    }
    float mine = 0;
    for (int s = 0; s < cut.splits; ++s) mine += sums[s * next + chosen];
    const float g = gate_of(rule, k, mine, most, all);
    if (lane < k) {
        A.idx[t * k + lane] = chosen;
        A.gate[t * k + lane] = g;
    }
}

// ---- the backward pass ----

// dl of a row, bf16, zeros from E to ld (a multiple of 8).
template <int Each>
__global__ __launch_bounds__(kChooseWaves * kWave) void router_dlogits_kernel(RouterShape S, Rule rule,
                                                                              const float* grad_gate,
                                                                              const float* logits, const int32_t* idx,
                                                                              const float* grad_logits,
                                                                              unsigned short* dl, int ld, GridSpan span)
{
    __shared__ float ds[kChooseWaves][Each * kWave];
    const int lane = lane_id(), E = S.E, k = S.k;
    const int64_t t = (int64_t)span_block(span) * kChooseWaves + wave_id();
    if (t >= S.T) return;
    float* const mine = ds[wave_id()];
#pragma unroll
    for (int i = 0; i < Each; ++i) mine[lane + i * kWave] = 0;
    float l[Each], most = -__builtin_inff(), all = 0;
#pragma unroll
    for (int i = 0; i < Each; ++i) {
        const int e = lane + i * kWave;
        l[i] = e < E ? logits[t * E + e] : -__builtin_inff();
        most = fmaxf(most, l[i]);
    }
    if (!rule.sigmoid) {
        most = wave_max(most);
#pragma unroll
        for (int i = 0; i < Each; ++i)
            if (lane + i * kWave < E) all += expf(l[i] - most);
        all = wave_total(all);
    }
    const auto score = [&](float v) { return rule.sigmoid ? 1.0f / (1.0f + expf(-v)) : expf(v - most) / all; };
    const int e = lane < k ? idx[t * k + lane] : 0;
    const bool in = lane < k && e >= 0 && e < E;
    const float s = in ? score(logits[t * E + e]) : 0.0f;
    float g = in ? rule.scale * grad_gate[t * k + lane] : 0.0f;
    if (rule.normalize) {
        const float total = wave_total(s) + 1e-20f;
        g = (g - wave_total(g * s) / total) / total;
        if (!in) g = 0.0f;
    }
    const float mean = rule.sigmoid ? 0.0f : wave_total(g * s);
    if (in) mine[e] = g;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's own LDS
#pragma unroll
    for (int i = 0; i < Each; ++i) {
        const int e = lane + i * kWave;
        if (e >= ld) continue;
        float d = 0;
        if (e < E) {
            const float g = mine[e];
            if (rule.sigmoid) {
                // 0 where nothing was chosen, also beside a logit that is not finite
                if (g != 0.0f) {
                    const float s = score(l[i]);
                    d = g * s * (1.0f - s);
                }
            } else {
                d = score(l[i]) * (g - mean);
            }
            if (grad_logits) d += grad_logits[t * E + e];
        }
        dl[t * ld + e] = (unsigned short)bf16_pack2(d, d);
    }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int64_t bytes)
{
    const uint64_t a = (uint64_t)p;  // the same in every lane
    const uint64_t q = (unsigned)__builtin_amdgcn_readfirstlane((int)a) |
                       (uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)(a >> 32)) << 32;
    return __builtin_amdgcn_make_buffer_rsrc((void*)q, 0, __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}

// grad_x = grad_x_in + dl W, a tile of rows and 256 columns a block.
template <bool Small>
__global__ __launch_bounds__(kGemmThreads, Small ? 4 : 2) void router_grad_x_kernel(RouterShape S, const char* dl, int ld,
                                                                                    const char* w, const char* in,
                                                                                    char* out, int across, GridSpan span)
{
    __shared__ __align__(1024) char lds[Lds<Small>::kBytes];
    const Place at = place_of(span, across);
    const int row0 = at.tile * Lds<Small>::kRows, nr = min(Lds<Small>::kRows, S.T - row0);
    if (nr <= 0) return;
    const int n0 = at.across * kTileFeatures, H = S.H, valid = min(H - n0, kTileFeatures), lane = lane_id();
    KContiguous r;
    r.init(ld, ld);
    KStrided f;
    f.init(H, S.E);
    for (int i = 0; i < 2; ++i) f.slot(i, w + (n0 + 128 * i) * 2, H - n0 - 128 * i);
    with_rows<Small>(nr, [&](auto mf) {
        constexpr int MF = decltype(mf)::value;
        Acc<MF> acc;
        row_slots<MF>(r, dl + (int64_t)row0 * ld * 2, ld, nr);
        tile_product<Small, MF>(r, f, S.E, lds, acc);
        const int64_t first = (int64_t)row0 * H + n0;
        const __amdgpu_buffer_rsrc_t add = buffer(in ? in + first * 2 : nullptr, in ? ((int64_t)nr * H - n0) * 2 : 0);
        write_tile<MF>(lds, nr, valid, out + first * 2, (int64_t)H * 2, [&](int m, int n) {
            const int row = row_of<MF>(m) + (lane & 15), c = feature_of(n) + 4 * (lane >> 4);
            // past the tile's rows and columns it is other rows' values or zero, and the sum goes nowhere
            const u32x2 d = __builtin_amdgcn_raw_buffer_load_b64(add, (unsigned)(row * H + c) * 2, 0, 0);
            const f32x4 v = acc[m][n];
            return pack4(f32x4{v[0] + bf16_lo(d[0]), v[1] + bf16_hi(d[0]), v[2] + bf16_lo(d[1]), v[3] + bf16_hi(d[1])});
        });
    });
}

// Part `blockIdx / tiles` of dl^T x: rows [part * each, ...) of both, 256 experts by 256 columns a block, fp32.
__global__ __launch_bounds__(kGemmThreads, 2) void router_grad_w_kernel(RouterShape S, const char* dl, int ld,
                                                                        const char* x, float* parts, int each, int splits,
                                                                        int across)
{
    __shared__ __align__(1024) char lds[Lds<false>::kBytes];
    // the parts vary fastest: the tiles of a part, which share dl, and those of neighbouring parts spread over the XCDs
    const int b = blockIdx.x, part = b % splits, tile = b / splits, e0 = tile / across * kTileRows;
    const int n0 = tile % across * kTileFeatures, H = S.H, E = S.E, lane = lane_id();
    const int64_t t0 = (int64_t)part * each;
    const int K = (int)min((int64_t)each, S.T - t0), nr = min(kTileRows, E - e0);
    KStrided r, f;
    r.init(ld, K);
    f.init(H, K);
    for (int i = 0; i < 2; ++i) f.slot(i, x + (t0 * H + n0 + 128 * i) * 2, H - n0 - 128 * i);
    with_rows<false>(nr, [&](auto mf) {
        constexpr int MF = decltype(mf)::value, kFirst = 32 * low_rows(MF);
        Acc<MF> acc;
        for (int i = 0; i < 2; ++i) r.slot(i, dl + (t0 * ld + e0 + kFirst * i) * 2, ld - e0 - kFirst * i);
        tile_product<false, MF>(r, f, K, lds, acc);
        // rows past the experts' last lie past the descriptor's end: nothing is written
        const __amdgpu_buffer_rsrc_t to = buffer(parts + ((int64_t)part * E + e0) * H + n0, ((int64_t)nr * H - n0) * 4);
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int row = row_of<MF>(m) + (lane & 15), c = feature_of(n) + 4 * (lane >> 4);
                if (n0 + c < H)
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[m][n]), to,
                                                           (unsigned)(row * H + c) * 4, 0, 0);
            }
    });
}

// bf16 of the parts' sum, eight elements a thread.
__global__ __launch_bounds__(256) void router_join_kernel(const f32x4* parts, int splits, int64_t vectors, u32x4* out)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= vectors) return;
    f32x4 a = {0, 0, 0, 0}, b = a;
    for (int s = 0; s < splits; ++s) {
        a += parts[(s * vectors + i) * 2];
        b += parts[(s * vectors + i) * 2 + 1];
    }
    out[i] = u32x4{bf16_pack2(a[0], a[1]), bf16_pack2(a[2], a[3]), bf16_pack2(b[0], b[1]), bf16_pack2(b[2], b[3])};
}

// ---- sizes ----

constexpr int kBlocks = 512;  // two small tiles a CU
constexpr int kMaxSplits = 16;

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

Cut cut_of(const RouterShape& S)
{
    const int64_t tiles = up(S.T, kTokens) * up(S.E, kTileFeatures);
    int splits = 1;
    // parts of at least four tiles of k, as long as there are fewer blocks than fill the card
    while (splits < kMaxSplits && tiles * splits * 2 <= kBlocks && S.H >= splits * 2 * 4 * kTileK) splits *= 2;
    Cut c;
    c.each = (int)up(up(S.H, splits), kTileK) * kTileK;
    c.splits = (int)up(S.H, c.each);
    c.ld = (int)up(S.E, 4) * 4;
    // roundings one after another: a matrix instruction for 32 k, the 32 products inside one, the sum of the parts
    c.gamma = (float)(c.each / 32 + 32 + c.splits + 8) * 1.1920929e-7f;
    return c;
}

struct GradCut {
    int splits, each, ld;
};

GradCut grad_cut(const RouterShape& S)
{
    const int64_t tiles = up(S.E, kTileRows) * up(S.H, kTileFeatures);
    int64_t splits = 256 / tiles;
    if (splits > up(S.T, 4 * kTileK)) splits = up(S.T, 4 * kTileK);
    if (splits > 32) splits = 32;
    if (splits < 1) splits = 1;
    GradCut c;
    c.each = (int)up(up(S.T, splits), kTileK) * kTileK;
    c.splits = (int)up(S.T, c.each);
    c.ld = (int)up(S.E, 8) * 8;
    return c;
}

hipError_t join(const float* parts, int splits, const RouterShape& S, void* grad_w, hipStream_t s)
{
    const int64_t vectors = (int64_t)S.E * S.H / 8;
    router_join_kernel<<<(unsigned)up(vectors, 256), 256, 0, s>>>((const f32x4*)parts, splits, vectors, (u32x4*)grad_w);
    return hipGetLastError();
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

template <template <int> class Go, class... Args>
hipError_t by_experts(int E, const Args&... args)
{
    if (E <= 64) return Go<1>::go(args...);
    if (E <= 128) return Go<2>::go(args...);
    if (E <= 256) return Go<4>::go(args...);
    return Go<16>::go(args...);
}

template <int Each>
struct GoChoose {
    static hipError_t go(const RouterShape& S, const Rule& rule, const Cut& cut, const Partial& P, const ChooseArgs& A,
                         hipStream_t s)
    {
        return launch_spans(up(S.T, kChooseWaves), kChooseWaves * kWave, [&](dim3 grid, GridSpan span) {
            router_choose_kernel<Each><<<grid, kChooseWaves * kWave, 0, s>>>(S, rule, cut, P, A, span);
        });
    }
};

template <int Each>
struct GoDlogits {
    static hipError_t go(const RouterShape& S, const Rule& rule, const float* grad_gate, const float* logits,
                         const int32_t* idx, const float* grad_logits, unsigned short* dl, int ld, hipStream_t s)
    {
        return launch_spans(up(S.T, kChooseWaves), kChooseWaves * kWave, [&](dim3 grid, GridSpan span) {
            router_dlogits_kernel<Each><<<grid, kChooseWaves * kWave, 0, s>>>(S, rule, grad_gate, logits, idx, grad_logits,
                                                                              dl, ld, span);
        });
    }
};

}  // namespace

size_t router_workspace(const RouterShape& S, bool backward)
{
    size_t n = 256;
    if (S.T > 0) {
        const Cut c = cut_of(S);
        n = align256((size_t)c.splits * S.T * c.ld * 4) + align256((size_t)c.splits * S.T * 4) +
            align256((size_t)c.splits * S.E * 4);
    }
    if (backward && S.T > 0) {
        const GradCut g = grad_cut(S);
        const size_t b = align256((size_t)S.T * g.ld * 2) + align256((size_t)g.splits * S.E * S.H * 4);
        if (b > n) n = b;
    }
    return n;
}

hipError_t launch_router_forward(const RouterShape& S, const Rule& rule, const void* x, const void* w, int32_t* idx,
                                 float* gate, float* logits, char* ws, hipStream_t s)
{
    const Cut cut = cut_of(S);
    Partial P;
    P.sum = (float*)ws;
    P.x2 = (float*)(ws + align256((size_t)cut.splits * S.T * cut.ld * 4));
    P.w2 = (float*)((char*)P.x2 + align256((size_t)cut.splits * S.T * 4));
    const int tiles = (int)up(S.T, kTokens);
    const int64_t grid = (int64_t)tiles * up(S.E, kTileFeatures) * cut.splits;
    const hipError_t e = launch_spans(grid, kGemmThreads, [&](dim3 blocks, GridSpan span) {
        router_logits_kernel<<<blocks, kGemmThreads, 0, s>>>(S, cut, P, (const char*)x, (const char*)w, tiles, span);
    });
    if (e != hipSuccess) return e;
    return by_experts<GoChoose>(S.E, S, rule, cut, P, ChooseArgs{(const u32x4*)x, (const u32x4*)w, idx, gate, logits}, s);
}

hipError_t launch_router_backward(const RouterShape& S, const Rule& rule, const float* grad_gate, const float* logits,
                                  const int32_t* idx, const void* x, const void* w, const float* grad_logits,
                                  const void* grad_x_in, void* grad_x, void* grad_w, char* ws, hipStream_t s)
{
    const GradCut g = S.T ? grad_cut(S) : GradCut{};
    unsigned short* const dl = (unsigned short*)ws;
    float* const parts = (float*)(ws + align256((size_t)S.T * g.ld * 2));
    if (S.T == 0)  // no part: zeros
        return grad_w ? join(parts, 0, S, grad_w, s) : hipSuccess;
    hipError_t e = by_experts<GoDlogits>(S.E, S, rule, grad_gate, logits, idx, grad_logits, dl, g.ld, s);
    if (e == hipSuccess && grad_x) {
        const int across = (int)up(S.H, kTileFeatures);
        e = launch_spans(places(up(S.T, Lds<true>::kRows), across), kGemmThreads, [&](dim3 grid, GridSpan span) {
            router_grad_x_kernel<true><<<grid, kGemmThreads, 0, s>>>(S, (const char*)dl, g.ld, (const char*)w,
                                                                     (const char*)grad_x_in, (char*)grad_x, across, span);
        });
    }
    if (e == hipSuccess && grad_w) {
        const int across = (int)up(S.H, kTileFeatures);
        const int64_t grid = up(S.E, kTileRows) * across * g.splits;
        router_grad_w_kernel<<<(unsigned)grid, kGemmThreads, 0, s>>>(S, (const char*)dl, g.ld, (const char*)x, parts, g.each,
                                                                     g.splits, across);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        e = join(parts, g.splits, S, grad_w, s);
    }
    return e;
}

}  // namespace ms
