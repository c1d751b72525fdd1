// experts_ffn.hip -- the matrix products of the experts' gated block.
#include "experts.h"

namespace ms {
namespace {

constexpr int kT = 64;   // rows and features of a tile
constexpr int kK = 32;   // its step along the sum
constexpr int kPad = 8;

struct Operand {
    const unsigned short* p;  // element (i, k) at p[i * si + k * sk]
    int64_t si, sk;
};

// acc[f] of wave w: rows 16 w .. + 16 (lane & 15), features 16 f + 4 (lane >> 4) .. + 4.
// Operand rows at or past nr, features whose index `feat` gives as -1, and k >= K count as zero.
template <class Feat>
__device__ __forceinline__ void tile_product(const Operand& R, int nr, const Operand& F, Feat feat, int K,
                                             unsigned short* sr, unsigned short* sf, f32x4 acc[4])
{
    const int lane = lane_id(), w = threadIdx.x >> 6;
    for (int f = 0; f < 4; ++f) acc[f] = f32x4{0, 0, 0, 0};
    for (int k0 = 0; k0 < K; k0 += kK) {
        __syncthreads();
        for (int i = threadIdx.x; i < kT * kK; i += 256) {
            const int r = R.sk == 1 ? i / kK : i % kT, k = R.sk == 1 ? i % kK : i / kT;
            sr[r * (kK + kPad) + k] = r < nr && k0 + k < K ? R.p[r * R.si + (k0 + k) * R.sk] : 0;
        }
        for (int i = threadIdx.x; i < kT * kK; i += 256) {
            const int n = F.sk == 1 ? i / kK : i % kT, k = F.sk == 1 ? i % kK : i / kT;
            const int f = feat(n);
            sf[n * (kK + kPad) + k] = f >= 0 && k0 + k < K ? F.p[f * F.si + (k0 + k) * F.sk] : 0;
        }
        __syncthreads();
        const bf16x8 b = *(const bf16x8*)(sr + (16 * w + (lane & 15)) * (kK + kPad) + 8 * (lane >> 4));
        for (int f = 0; f < 4; ++f) {
            const bf16x8 a = *(const bf16x8*)(sf + (16 * f + (lane & 15)) * (kK + kPad) + 8 * (lane >> 4));
            acc[f] = mfma_16x16x32(a, b, acc[f]);
        }
    }
}

__device__ __forceinline__ void store4(void* p, int64_t at, f32x4 v)
{
    *(u32x2*)((unsigned short*)p + at) = u32x2{bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3])};
}

__device__ __forceinline__ f32x4 load4(const void* p, int64_t at)
{
    const u32x2 u = *(const u32x2*)((const unsigned short*)p + at);
    return f32x4{bf16_lo(u[0]), bf16_hi(u[0]), bf16_lo(u[1]), bf16_hi(u[1])};
}

// Largest magnitude over the 32 features that the four lanes of a row hold in
// v[0] and v[1]; infinity if any is not finite.
__device__ __forceinline__ float group_top(f32x4 a, f32x4 b)
{
    float top = 0;
    bool bad = false;
    for (int i = 0; i < 4; ++i) {
        top = fmaxf(top, fmaxf(fabsf(a[i]), fabsf(b[i])));
        bad |= !(fabsf(a[i]) <= 3.40282347e38f) || !(fabsf(b[i]) <= 3.40282347e38f);
    }
    if (bad) top = __uint_as_float(0x7f800000u);
    top = fmaxf(top, __shfl_xor(top, 16, kWave));
    return fmaxf(top, __shfl_xor(top, 32, kWave));
}

__global__ __launch_bounds__(256) void ffn_up_kernel(ExpertShape S, const unsigned short* xe, const unsigned short* w,
                                                     void* h, SavedActs saved)
{
    __shared__ __align__(16) unsigned short sr[kT * (kK + kPad)], sf[kT * (kK + kPad)];
    if (*S.status) return;
    int r0, nr;
    const int e = segment_tile(S.offset, S.E, kT, 16, blockIdx.x, &r0, &nr);
    if (e < 0) return;
    const int c0 = blockIdx.y * 32;
    f32x4 acc[4];
    const Operand R{xe + (int64_t)r0 * S.H, S.H, 1}, F{w + (int64_t)e * 2 * S.I * S.H, S.H, 1};
    const int I = S.I;
    tile_product(R, nr, F, [=](int n) { const int c = c0 + (n & 31); return c < I ? (n < 32 ? c : I + c) : -1; }, S.H,
                 sr, sf, acc);
    const int lane = lane_id(), r = 16 * (threadIdx.x >> 6) + (lane & 15);
    const int64_t row = r0 + r;
    const bool ok = r < nr;
    for (int i = 0; i < 2; ++i) {
        const int c = c0 + 16 * i + 4 * (lane >> 4);
        f32x4 v;
        for (int j = 0; j < 4; ++j) {
            float slope;
            v[j] = acc[i][j] * gate_sigmoid(acc[i][j], S.c0, S.c1, &slope) * acc[2 + i][j];
        }
        if (ok && c < I) {
            store4(h, row * I + c, v);
            if (saved.data && !saved.scale) {
                store4(saved.data, row * 2 * I + c, acc[i]);
                store4(saved.data, row * 2 * I + I + c, acc[2 + i]);
            }
        }
    }
    if (saved.scale) {
        const int groups = (I + kGroup8 - 1) / kGroup8;
        for (int which = 0; which < 2; ++which) {
            const float step = step8(group_top(acc[2 * which], acc[2 * which + 1])), inv = 1.0f / step;
            if (!ok) continue;
            for (int i = 0; i < 2; ++i) {
                const int c = c0 + 16 * i + 4 * (lane >> 4);
                const f32x4 v = acc[2 * which + i];
                if (c < I)
                    *(unsigned*)((char*)saved.data + row * 2 * I + which * I + c) = pack8x4(v[0], v[1], v[2], v[3], inv);
            }
            if (lane < 16)
                ((unsigned short*)saved.scale)[(row * 2 + which) * groups + blockIdx.y] =
                    (unsigned short)(__float_as_uint(step) >> 16);
        }
    }
}

// out[row] = R F^T for the rows of every expert: R [P, K] row-major, F of expert e at w + e * fe.
__global__ __launch_bounds__(256) void ffn_rows_kernel(ExpertShape S, const unsigned short* in, int K, Operand F,
                                                       int64_t fe, int N, void* out)
{
    __shared__ __align__(16) unsigned short sr[kT * (kK + kPad)], sf[kT * (kK + kPad)];
    if (*S.status) return;
    int r0, nr;
    const int e = segment_tile(S.offset, S.E, kT, 16, blockIdx.x, &r0, &nr);
    if (e < 0) return;
    f32x4 acc[4];
    F.p += e * fe;
    const int n0 = blockIdx.y * kT;
    tile_product(Operand{in + (int64_t)r0 * K, K, 1}, nr, F, [=](int n) { return n0 + n < N ? n0 + n : -1; }, K, sr,
                 sf, acc);
    const int lane = lane_id(), r = 16 * (threadIdx.x >> 6) + (lane & 15);
    for (int f = 0; f < 4; ++f) {
        const int c = n0 + 16 * f + 4 * (lane >> 4);
        if (r < nr && c < N) store4(out, (int64_t)(r0 + r) * N + c, acc[f]);
    }
}

__global__ __launch_bounds__(256) void ffn_dh_kernel(ExpertShape S, const unsigned short* gy, const unsigned short* w,
                                                     SavedActs saved, void* h, void* dgu)
{
    __shared__ __align__(16) unsigned short sr[kT * (kK + kPad)], sf[kT * (kK + kPad)];
    if (*S.status) return;
    int r0, nr;
    const int e = segment_tile(S.offset, S.E, kT, 16, blockIdx.x, &r0, &nr);
    if (e < 0) return;
    f32x4 acc[4];
    const int n0 = blockIdx.y * kT, I = S.I;
    tile_product(Operand{gy + (int64_t)r0 * S.H, S.H, 1}, nr, Operand{w + (int64_t)e * S.H * I, 1, I},
                 [=](int n) { return n0 + n < I ? n0 + n : -1; }, S.H, sr, sf, acc);
    const int lane = lane_id(), r = 16 * (threadIdx.x >> 6) + (lane & 15);
    const int64_t row = r0 + r;
    const int groups = (I + kGroup8 - 1) / kGroup8;
    for (int f = 0; f < 4; ++f) {
        const int c = n0 + 16 * f + 4 * (lane >> 4);
        if (r >= nr || c >= I) continue;
        f32x4 g, u;
        if (saved.scale) {
            const unsigned short* sc = (const unsigned short*)saved.scale + row * 2 * groups + c / kGroup8;
            const float sg = __uint_as_float((unsigned)sc[0] << 16), su = __uint_as_float((unsigned)sc[groups] << 16);
            const unsigned qg = *(const unsigned*)((const char*)saved.data + row * 2 * I + c);
            const unsigned qu = *(const unsigned*)((const char*)saved.data + row * 2 * I + I + c);
            for (int j = 0; j < 4; ++j) { g[j] = int8_of(qg, j) * sg; u[j] = int8_of(qu, j) * su; }
        } else {
            g = load4(saved.data, row * 2 * I + c);
            u = load4(saved.data, row * 2 * I + I + c);
        }
        f32x4 dg, du, hv;
        for (int j = 0; j < 4; ++j) {
            float slope;
            const float s = gate_sigmoid(g[j], S.c0, S.c1, &slope), a = g[j] * s;
            hv[j] = a * u[j];
            du[j] = acc[f][j] * a;
            dg[j] = acc[f][j] * u[j] * fmaf(a * (1.0f - s), slope, s);
        }
        store4(h, row * I + c, hv);
        store4(dgu, row * 2 * I + c, dg);
        store4(dgu, row * 2 * I + I + c, du);
    }
}

__global__ __launch_bounds__(256) void ffn_wgrad_kernel(ExpertShape S, const unsigned short* a, int na,
                                                        const unsigned short* b, int nb, void* out)
{
    __shared__ __align__(16) unsigned short sr[kT * (kK + kPad)], sf[kT * (kK + kPad)];
    if (*S.status) return;
    const int tm = (na + kT - 1) / kT;
    const int e = blockIdx.x / tm, m0 = (blockIdx.x % tm) * kT, n0 = blockIdx.y * kT;
    const int q0 = S.offset[e], rows = S.offset[e + 1] - q0;
    f32x4 acc[4];
    tile_product(Operand{a + (int64_t)q0 * na + m0, 1, na}, na - m0, Operand{b + (int64_t)q0 * nb, 1, nb},
                 [=](int n) { return n0 + n < nb ? n0 + n : -1; }, rows, sr, sf, acc);
    const int lane = lane_id(), m = m0 + 16 * (threadIdx.x >> 6) + (lane & 15);
    for (int f = 0; f < 4; ++f) {
        const int c = n0 + 16 * f + 4 * (lane >> 4);
        if (m < na && c < nb) store4(out, ((int64_t)e * na + m) * nb + c, acc[f]);
    }
}

int row_tiles(const ExpertShape& S) { return S.P / kT + (S.P < S.E ? S.P : S.E); }

}  // namespace

hipError_t launch_ffn_up(const ExpertShape& S, const void* xe, const void* w_gate_up, void* h, SavedActs saved,
                         hipStream_t s)
{
    ffn_up_kernel<<<dim3(row_tiles(S), (S.I + 31) / 32), 256, 0, s>>>(S, (const unsigned short*)xe,
                                                                      (const unsigned short*)w_gate_up, h, saved);
    return hipGetLastError();
}

hipError_t launch_ffn_down(const ExpertShape& S, const void* h, const void* w_down, void* ye, hipStream_t s)
{
    ffn_rows_kernel<<<dim3(row_tiles(S), (S.H + kT - 1) / kT), 256, 0, s>>>(
        S, (const unsigned short*)h, S.I, Operand{(const unsigned short*)w_down, S.I, 1}, (int64_t)S.H * S.I, S.H, ye);
    return hipGetLastError();
}

hipError_t launch_ffn_dh(const ExpertShape& S, const void* grad_ye, const void* w_down, SavedActs saved, void* h,
                         void* dgu, hipStream_t s)
{
    ffn_dh_kernel<<<dim3(row_tiles(S), (S.I + kT - 1) / kT), 256, 0, s>>>(
        S, (const unsigned short*)grad_ye, (const unsigned short*)w_down, saved, h, dgu);
    return hipGetLastError();
}

hipError_t launch_ffn_dx(const ExpertShape& S, const void* dgu, const void* w_gate_up, void* grad_xe, hipStream_t s)
{
    ffn_rows_kernel<<<dim3(row_tiles(S), (S.H + kT - 1) / kT), 256, 0, s>>>(
        S, (const unsigned short*)dgu, 2 * S.I, Operand{(const unsigned short*)w_gate_up, 1, S.H},
        (int64_t)2 * S.I * S.H, S.H, grad_xe);
    return hipGetLastError();
}

hipError_t launch_ffn_wgrad(const ExpertShape& S, const void* a, int na, const void* b, int nb, void* out,
                            hipStream_t s)
{
    ffn_wgrad_kernel<<<dim3(S.E * ((na + kT - 1) / kT), (nb + kT - 1) / kT), 256, 0, s>>>(
        S, (const unsigned short*)a, na, (const unsigned short*)b, nb, out);
    return hipGetLastError();
}

}  // namespace ms
