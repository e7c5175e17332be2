// Root-mean-square norm with the residual's addition, written in bf16 and / or
// in int8 with one scale per row (what qgemm_skinny_run's 8-bit format reads),
// optionally rotated by the block-diagonal randomized Hadamard-32.
//
//   r = x + residual;  rs = 1 / sqrt(mean r^2 + eps);  y = r rs w
//   z = r w, or H32 (d . r w) in each block of 32 with the signs d
//   Xq = round-half-even(z * 127 / max|z|),  x_scales = max|z| rs / 127
//        (/ sqrt(32) when rotated)
// The codes do not depend on rs.  They are decided in fp64 (like
// hadamard32_quant_run's), where r w of bf16 inputs is exact, so they are the
// definition's codes whatever the order of the sums; r for y and the sum of
// squares are fp32.
//
// One workgroup per row; a thread holds U units of 8 consecutive elements, the
// four lanes of a quad one block of 32.
#include "rmsnorm.h"

namespace qg {

namespace {

template <int S>
__device__ __forceinline__ double quad_xor(double v) {
    constexpr int ctrl = S == 1 ? 0xB1 : 0x4E;  // [1,0,3,2] / [2,3,0,1]
    const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
    const int lo = __builtin_amdgcn_mov_dpp((int)(unsigned)u, ctrl, 0xF, 0xF, false);
    const int hi = __builtin_amdgcn_mov_dpp((int)(unsigned)(u >> 32), ctrl, 0xF, 0xF, false);
    return __builtin_bit_cast(double, ((unsigned long long)(unsigned)hi << 32) | (unsigned)lo);
}

// z <- H32 z over the quad's block; lane part p holds elements 8p .. 8p+7
__device__ __forceinline__ void fwht32(double z[8], int p) {
#pragma unroll
    for (int s = 1; s < 8; s <<= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (!(e & s)) {
                const double a = z[e], c = z[e + s];
                z[e] = a + c;
                z[e + s] = a - c;
            }
    const double sg1 = (p & 1) ? -1.0 : 1.0, sg2 = (p & 2) ? -1.0 : 1.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = fma(z[e], sg1, quad_xor<1>(z[e]));
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = fma(z[e], sg2, quad_xor<2>(z[e]));
}

// 8 values of a bf16 or fp32 row
template <bool F32>
__device__ __forceinline__ void load8(const void *row, int unit, float v[8]) {
    if (F32) {
        const f32x4_t *p = reinterpret_cast<const f32x4_t *>(row) + 2 * unit;
        const f32x4_t a = p[0], b = p[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = a[e];
            v[4 + e] = b[e];
        }
    } else {
        const u32x4_t a = reinterpret_cast<const u32x4_t *>(row)[unit];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = bf16_lo(a[e]);
            v[2 * e + 1] = bf16_hi(a[e]);
        }
    }
}

__device__ __forceinline__ u32x4_t pack_bf16(const float v[8]) {
    u32x4_t o;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        o[e] = (unsigned)f32_to_bf16(v[2 * e]) | ((unsigned)f32_to_bf16(v[2 * e + 1]) << 16);
    return o;
}

}  // namespace

// RES: 0 none, 1 bf16, 2 fp32
template <int U, bool XF32, int RES, bool Q, bool ROT>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(RmsArgs a) {
    __shared__ float wss[16];
    __shared__ double wmax[16];
    const size_t m = blockIdx.x;
    const int tid = threadIdx.x, nt = blockDim.x, nw = nt >> 6;
    const int units = a.K >> 3;
    const size_t row = m * (size_t)a.K;
    const char *x = reinterpret_cast<const char *>(a.x) + row * (XF32 ? 4 : 2);
    const char *res = reinterpret_cast<const char *>(a.residual) + row * (RES == 2 ? 4 : 2);
    float r[U][8];
    double z[Q ? U : 1][8];
    float ss = 0.f;
    double amax = 0.0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = tid + i * nt;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] = 0.f;
        if (u < units) {  // uniform over a quad: K is a multiple of 32
            float xv[8], rv[8];
            load8<XF32>(x, u, xv);
            if (RES) load8<RES == 2>(res, u, rv);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                r[i][e] = RES ? xv[e] + rv[e] : xv[e];
                ss = fmaf(r[i][e], r[i][e], ss);
            }
            if (RES && a.residual_out) {
                char *out = reinterpret_cast<char *>(a.residual_out) + row * (RES == 2 ? 4 : 2);
                if (RES == 2) {
                    f32x4_t *o = reinterpret_cast<f32x4_t *>(out) + 2 * u;
                    o[0] = f32x4_t{r[i][0], r[i][1], r[i][2], r[i][3]};
                    o[1] = f32x4_t{r[i][4], r[i][5], r[i][6], r[i][7]};
                } else {
                    reinterpret_cast<u32x4_t *>(out)[u] = pack_bf16(r[i]);
                }
            }
            if (Q) {
                float w[8];
                load8<false>(a.weight, u, w);
                u32x2_t sg = {0u, 0u};
                if (ROT) sg = reinterpret_cast<const u32x2_t *>(a.signs)[u];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    double v = RES ? (double)xv[e] + (double)rv[e] : (double)xv[e];
                    v *= (double)w[e];
                    if (ROT) v *= (double)(int8_t)((sg[e >> 2] >> (8 * (e & 3))) & 0xFFu);
                    z[i][e] = v;
                }
                if (ROT) fwht32(z[i], tid & 3);
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmax(amax, fabs(z[i][e]));
            }
        }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        ss += __shfl_xor(ss, d);
        if (Q) amax = fmax(amax, __shfl_xor(amax, d));
    }
    if ((tid & 63) == 0) {
        wss[tid >> 6] = ss;
        if (Q) wmax[tid >> 6] = amax;
    }
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < nw; ++w) {
        ss += wss[w];
        if (Q) amax = fmax(amax, wmax[w]);
    }
    const float rs = 1.f / sqrtf(ss / (float)a.K + a.eps);
    // a row with a NaN or an infinity has no scale: codes 0, scale NaN
    const bool fin = ss < __builtin_inff();
    const double f = fin && amax > 0.0 ? 127.0 / amax : 0.0;
    if (Q && tid == 0)
        a.x_scales[m] = !fin         ? __builtin_nanf("")
                        : amax > 0.0 ? (float)(amax * (double)rs / a.denom)
                                     : 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = tid + i * nt;
        if (u >= units) continue;
        if (a.y) {
            float w[8], v[8];
            load8<false>(a.weight, u, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = r[i][e] * rs * w[e];
            reinterpret_cast<u32x4_t *>(a.y + row)[u] = pack_bf16(v);
        }
        if (Q) {
            unsigned packed[2] = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // the quotient itself where its approximation is near a border
                const double p = z[i][e] * f;
                double q = rint(p);
                if (fabs(p - q) > 0.5 - 1e-9) q = rint(z[i][e] * 127.0 / amax);
                packed[e >> 2] |= ((unsigned)(int)(fin ? q : 0.0) & 0xFFu) << (8 * (e & 3));
            }
            *reinterpret_cast<u32x2_t *>(a.Xq + row + 8 * u) = u32x2_t{packed[0], packed[1]};
        }
    }
}

namespace {

template <int U, bool XF32, int RES>
void run(const RmsArgs &a, int threads, hipStream_t s) {
    const dim3 g((unsigned)a.M), b(threads);
    if (!a.Xq)
        hipLaunchKernelGGL((rmsnorm_kernel<U, XF32, RES, false, false>), g, b, 0, s, a);
    else if (!a.signs)
        hipLaunchKernelGGL((rmsnorm_kernel<U, XF32, RES, true, false>), g, b, 0, s, a);
    else
        hipLaunchKernelGGL((rmsnorm_kernel<U, XF32, RES, true, true>), g, b, 0, s, a);
}

template <int U>
void pick(const RmsArgs &a, bool xf32, int res, int threads, hipStream_t s) {
    if (xf32)
        res == 0 ? run<U, true, 0>(a, threads, s) : res == 1 ? run<U, true, 1>(a, threads, s) : run<U, true, 2>(a, threads, s);
    else
        res == 0 ? run<U, false, 0>(a, threads, s) : res == 1 ? run<U, false, 1>(a, threads, s) : run<U, false, 2>(a, threads, s);
}

}  // namespace

hipError_t launch_rmsnorm(const RmsArgs &a, bool x_f32, int res, hipStream_t s) {
    const int units = a.K / 8;
    const int u = units <= 1024 ? 1 : 3;
    const int threads = (((units + u - 1) / u) + 63) / 64 * 64;
    if (u == 1)
        pick<1>(a, x_f32, res, threads, s);
    else
        pick<3>(a, x_f32, res, threads, s);
    return hipGetLastError();
}

}  // namespace qg
