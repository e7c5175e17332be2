// Root-mean-square norm with the residual's addition, written in bf16 and / or
// in int8 with one scale per row (what qgemm_skinny_run's 8-bit format reads),
// optionally rotated by the block-diagonal randomized Hadamard-32.
//
//   r = x + residual;  rs = 1 / sqrt(mean r^2 + eps);  y = r rs w
//   z = r w, or H32 (d . r w) in each block of 32 with the signs d
//   Xq = round-half-even(z * 127 / max|z|),  x_scales = max|z| rs / 127
//        (/ sqrt(32) when rotated)
// The codes do not depend on rs.  They are the definition's codes whatever the
// order of the sums: z and max |z| count as fp64 has them (like
// hadamard32_quant_run's), where r w of bf16 inputs is exact.  Rotated, z is
// carried in fp64.  Otherwise fp32 decides, except where its value p (of four
// roundings, so off by at most 4 * 2^-24 |p| < 2.5e-7 |p|) is that near a
// border: that element is computed again in fp64 from its inputs.  So are,
// for max |z|, the elements within 2^-21 of fp32's largest, and all elements of
// a row whose largest product fp32 has below 2^-60 or as infinite.  r for y and
// the sum of squares are fp32.
//
// One workgroup per row; a thread holds U units of 8 consecutive elements, the
// four lanes of a quad one block of 32.  Bound by latency for a few rows (2.4
// us for 1 x 4096 in bf16, 6.8 for 32 x 12288 in fp32, rotated), by memory for
// many (5003 x 7168, residual, bf16 and codes: 67 us, 4.8 TB/s; in bf16 alone
// 54 us, 5.3 TB/s).  With every element in fp64 that took 85 us, with a border
// of 1e-4 codes 104: an element computed again waits for memory.
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
        o[e] = __builtin_bit_cast(unsigned, bf16x2_t{(__bf16)v[2 * e], (__bf16)v[2 * e + 1]});
    return o;
}

// element k of a row
template <bool F32>
__device__ __forceinline__ double load1(const void *row, int k) {
    if (F32) return (double)reinterpret_cast<const float *>(row)[k];
    return (double)bf16_lo(reinterpret_cast<const uint16_t *>(row)[k]);
}

}  // namespace

// RES: 0 none, 1 bf16, 2 fp32
template <int U, bool XF32, int RES, bool Q, bool ROT>
__global__ void __launch_bounds__(U == 4 ? 256 : 1024) rmsnorm_kernel(RmsArgs a) {
    __shared__ float wss[16];
    __shared__ double wmax[16];
    __shared__ unsigned long long top_bits;
    const size_t m = blockIdx.x;
    const int tid = threadIdx.x, nt = blockDim.x, nw = nt >> 6;
    const int units = a.K >> 3;
    const size_t row = m * (size_t)a.K;
    const char *x = reinterpret_cast<const char *>(a.x) + row * (XF32 ? 4 : 2);
    const char *res = reinterpret_cast<const char *>(a.residual) + row * (RES == 2 ? 4 : 2);
    float r[U][8];
    u32x4_t wt[U];
    double z[ROT ? U : 1][8];
    float ss = 0.f;
    double amax = 0.0;
    if (Q && !ROT && tid == 0) top_bits = 0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = tid + i * nt;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] = 0.f;
        wt[i] = u32x4_t{0u, 0u, 0u, 0u};
        if (ROT)
#pragma unroll
            for (int e = 0; e < 8; ++e) z[i][e] = 0.0;
        if (u < units) {  // uniform over a quad: K is a multiple of 32
            float xv[8], rv[8];
            load8<XF32>(x, u, xv);
            if (RES) load8<RES == 2>(res, u, rv);
            wt[i] = reinterpret_cast<const u32x4_t *>(a.weight)[u];
            u32x2_t sg = {0u, 0u};
            if (ROT) sg = reinterpret_cast<const u32x2_t *>(a.signs)[u];
#pragma unroll
            for (int e = 0; e < 8; ++e) r[i][e] = RES ? xv[e] + rv[e] : xv[e];
            if (ROT) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float w = e & 1 ? bf16_hi(wt[i][e >> 1]) : bf16_lo(wt[i][e >> 1]);
                    z[i][e] = (RES ? (double)xv[e] + (double)rv[e] : (double)xv[e]) * (double)w *
                              (double)(int8_t)((sg[e >> 2] >> (8 * (e & 3))) & 0xFFu);
                }
                fwht32(z[i], tid & 3);
            }
        }
    }
    float zmax = 0.f;  // of fp32's r w
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ss = fmaf(r[i][e], r[i][e], ss);
            if (Q && ROT) amax = fmax(amax, fabs(z[i][e]));
            if (Q && !ROT) zmax = fmaxf(zmax, fabsf(r[i][e] * (e & 1 ? bf16_hi(wt[i][e >> 1]) : bf16_lo(wt[i][e >> 1]))));
        }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        ss += __shfl_xor(ss, d);
        if (Q && ROT) amax = fmax(amax, __shfl_xor(amax, d));
        if (Q && !ROT) zmax = fmaxf(zmax, __shfl_xor(zmax, d));
    }
    if ((tid & 63) == 0) {
        wss[tid >> 6] = ss;
        if (Q) wmax[tid >> 6] = ROT ? amax : (double)zmax;
    }
    __syncthreads();
    ss = 0.f;
    amax = 0.0;
    for (int w = 0; w < nw; ++w) {
        ss += wss[w];
        if (Q) amax = fmax(amax, wmax[w]);
    }
    // products this small have lost bits in fp32, or all of them, and some past
    // its range are infinite in it: fp64 decides every element
    const bool by64 = Q && !ROT && !(amax >= 0x1p-60 && amax < (double)__builtin_inff());
    bool nonzero = true;  // (a row of zeros needs none of that)
    if (by64) {
        unsigned any = 0u;
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) any |= __builtin_bit_cast(unsigned, r[i][e]) << 1;
        nonzero = __syncthreads_or(any != 0u);
    }
    // z in fp64 from its inputs (not rotated)
    const auto exact = [&](int k) {
        const double v = load1<XF32>(x, k);
        return (RES ? v + load1<RES == 2>(res, k) : v) * (double)bf16_lo(a.weight[k]);
    };
    const float rs = 1.f / sqrtf(ss / (float)a.K + a.eps);
    // a row with a NaN or an infinity has no scale: codes 0, scale NaN
    const bool fin = ss < __builtin_inff();
    if (Q && !ROT && fin && nonzero) {
        const float near = by64 ? 0.f : (float)amax * (1.f - 0x1p-21f);
        unsigned mine = 0u;  // the thread's elements that may be the largest
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                mine |= fabsf(r[i][e] * (e & 1 ? bf16_hi(wt[i][e >> 1]) : bf16_lo(wt[i][e >> 1]))) >= near ? 1u << (8 * i + e) : 0u;
#pragma unroll 1
        for (; mine; mine &= mine - 1) {
            const int k = __builtin_ctz(mine);
            if (tid + (k >> 3) * nt >= units) break;
            atomicMax(&top_bits, __builtin_bit_cast(unsigned long long, fabs(exact(8 * (tid + (k >> 3) * nt) + (k & 7)))));
        }
        __syncthreads();
        amax = __builtin_bit_cast(double, top_bits);
    }
    const double f = fin && amax > 0.0 ? 127.0 / amax : 0.0;
    const float f32 = (float)f;
    if (Q && tid == 0)
        a.x_scales[m] = !fin         ? __builtin_nanf("")
                        : amax > 0.0 ? (float)(amax * (double)rs / a.denom)
                                     : 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = tid + i * nt;
        if (u >= units) continue;
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = e & 1 ? bf16_hi(wt[i][e >> 1]) : bf16_lo(wt[i][e >> 1]);
        if (Q) {
            int q[8];
            unsigned border = 0u;  // elements near one
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (ROT) {
                    // the quotient itself where its approximation is near a border
                    const double p = z[i][e] * f;
                    double c = rint(p);
                    if (fabs(p - c) > 0.5 - 1e-9) c = rint(z[i][e] * 127.0 / amax);
                    q[e] = (int)c;
                } else {
                    const float p = r[i][e] * w[e] * f32, c = rintf(p);
                    border |= fabsf(p - c) > fmaf(fabsf(p), -2.5e-7f, 0.5f) ? 1u << e : 0u;
                    q[e] = (int)c;
                }
            }
            u32x2_t o = {(q[0] & 0xFFu) | (q[1] & 0xFFu) << 8 | (q[2] & 0xFFu) << 16 | (unsigned)q[3] << 24,
                         (q[4] & 0xFFu) | (q[5] & 0xFFu) << 8 | (q[6] & 0xFFu) << 16 | (unsigned)q[7] << 24};
            if (by64) border = 0xFFu;
            if (!fin || !(amax > 0.0)) {
                o = u32x2_t{0u, 0u};
                border = 0u;
            }
#pragma unroll 1
            for (; border; border &= border - 1) {
                const int e = __builtin_ctz(border), sh = 8 * (e & 3);
                const unsigned c = (unsigned)(int)rint(exact(8 * u + e) * 127.0 / amax) & 0xFFu;
                if (e < 4)
                    o[0] = (o[0] & ~(0xFFu << sh)) | c << sh;
                else
                    o[1] = (o[1] & ~(0xFFu << sh)) | c << sh;
            }
            *reinterpret_cast<u32x2_t *>(a.Xq + row + 8 * u) = o;
        }
        if (a.y) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = r[i][e] * rs * w[e];
            reinterpret_cast<u32x4_t *>(a.y + row)[u] = pack_bf16(v);
        }
        // last: it may take the residual's place, which the lines above read
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
    }
}

namespace {

template <int U, bool XF32, int RES>
void run(const RmsArgs &a, int threads, hipStream_t s) {
    const dim3 g((unsigned)a.M), b(threads);
    if constexpr (U != 4)
        if (!a.Xq) {
            hipLaunchKernelGGL((rmsnorm_kernel<U, XF32, RES, false, false>), g, b, 0, s, a);
            return;
        }
    if (!a.signs)
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
    // One unit a thread while 1024 threads take the row.  Not where codes are
    // asked of many rows of 9 waves or more: the codes wait for two reductions
    // of the whole workgroup, and too few of these are on a CU to hide that
    // (4 units against 1: 67.6 us against 74.0 for 5003 x 7168, but 63.9
    // against 58.2 for 8192 x 4096, 5.7 against 5.2 for 32 x 7168 and, in bf16
    // alone, 59.1 against 54.4 for 5003 x 7168).
    const int units = a.K / 8;
    const int u = units > 1024 ? 3 : a.Xq && a.M >= 512 && units > 512 ? 4 : 1;
    const int threads = (((units + u - 1) / u) + 63) / 64 * 64;
    if (u == 1)
        pick<1>(a, x_f32, res, threads, s);
    else if (u == 3)
        pick<3>(a, x_f32, res, threads, s);
    else
        pick<4>(a, x_f32, res, threads, s);
    return hipGetLastError();
}

}  // namespace qg
