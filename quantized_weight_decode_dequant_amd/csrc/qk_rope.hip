// Root-mean-square norm of each query and key head, with the position
// rotation in the same pass.
//
//   y = x w / sqrt(mean x^2 + eps)            over a head's D dimensions
//   angle_i = position[axis_i] * inv_freq_i   for each of `half` pairs
//   (a, b) -> (a cos - b sin, b cos + a sin)  pairs (i, i + half) or (2i, 2i + 1)
//
// The angle is an fp64 product in turns (two roundings, 2^-52 of it) reduced to
// half a turn there, so a position of 2^30 is nearly as good as one of 10;
// its sine and cosine, the norm and the rotation are fp32, and the one
// rounding to fewer bits is the output's to bf16.
//
// A wave takes heads of one token: LG lanes a head, 8 dimensions (16 bytes of
// bf16) a lane, U groups of 64 / LG heads in flight.  Its lanes make one
// angle each (two or four of wide heads) while the first heads are on their
// way, and pass them on through LDS.  Few tokens are split over several waves
// of as few heads as one load takes (`parts`), many take one wave each.
//
// Bound by latency for few tokens (1 of 32 + 8 heads of 128: 3.6 us, where an
// empty launch takes 2.4; 32 fp32 tokens on three axes 4.3), by memory for
// many (5003 tokens 24 us, 4.3 TB/s; 1021 of 32 + 4 heads of 256, a quarter
// rotated, no norm: 9.9 us, 3.8 TB/s).
#include "qk_rope.h"

namespace qg {

namespace {

// one lane's 8 values, as loaded
template <bool F32>
struct Raw {
    u32x4_t v[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Raw<F32> load_raw(const void *base, size_t at) {
    Raw<F32> r;
    if constexpr (F32) {
        const u32x4_t *p = reinterpret_cast<const u32x4_t *>((const float *)base + at);
        r.v[0] = p[0];
        r.v[1] = p[1];
    } else {
        r.v[0] = *reinterpret_cast<const u32x4_t *>((const uint16_t *)base + at);
    }
    return r;
}

__device__ __forceinline__ void bf16x8(u32x4_t w, float x[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16_lo(w[e]);
        x[2 * e + 1] = bf16_hi(w[e]);
    }
}

template <bool F32, bool INTERLEAVED, int LG>
__global__ void __launch_bounds__(256) qk_rope_kernel(QkRopeArgs a) {
    constexpr int HPL = 64 / LG;          // heads of one load
    constexpr int U = F32 ? 3 : 5;        // loads in flight
    constexpr int MAXH = LG * 4 > 64 ? LG * 4 : 64;
    __shared__ float cs[4][2][MAXH];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ul = lane % LG, hl = lane / LG, d = 8 * ul;
    const int64_t which = (int64_t)blockIdx.x * 4 + wave;  // (token, part of its heads)
    const int m = (int)(which / a.parts);
    const bool there = m < a.M;
    const int h0 = (int)(which % a.parts) * a.per_wave, h1 = there ? min(h0 + a.per_wave, a.H) : h0;
    const bool in = d < a.D;

    // the heads from h on, one load each
    Raw<F32> raw[U];
    const auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int hu = h + u * HPL + hl;
            if (hu < h1 && in) {
                const bool q = hu < a.Hq;
                raw[u] = load_raw<F32>(q ? a.q : a.k, q ? (size_t)m * a.q_stride + (size_t)hu * a.D + d
                                                        : (size_t)m * a.k_stride + (size_t)(hu - a.Hq) * a.D + d);
            } else {
                raw[u] = Raw<F32>{};
            }
        }
    };
    load(h0);
    float qw[8], kw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) qw[e] = kw[e] = 1.f;
    if (in && a.q_weight) bf16x8(*reinterpret_cast<const u32x4_t *>(a.q_weight + d), qw);
    if (in && a.k_weight) bf16x8(*reinterpret_cast<const u32x4_t *>(a.k_weight + d), kw);
    if (there) {
        for (int i = lane; i < a.half; i += 64) {
            const int ax = a.axis ? a.axis[i] : 0;
            const int pos = ax < a.axes ? a.positions[(size_t)ax * a.M + m] : 0;
            const double turns = (double)pos * ((double)a.inv_freq[i] * 0.15915494309189533577);
            float sn, c;
            sincospif(2.f * (float)(turns - rint(turns)), &sn, &c);
            cs[wave][0][i] = c;
            cs[wave][1][i] = sn;
        }
    }
    __syncthreads();
    if (!there) return;
    // the lane's angles: of its 8 dimensions, or its 4 pairs
    const int Dr = 2 * a.half, step = a.half / 8;
    const bool second = !INTERLEAVED && d >= a.half, turned = d < Dr;
    float c[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = INTERLEAVED ? (d + e) >> 1 : second ? d + e - a.half : d + e;
        c[e] = turned ? cs[wave][0][i] : 1.f;
        sn[e] = turned ? cs[wave][1][i] : 0.f;
        // the first of a pair takes its partner's sine negative
        if (INTERLEAVED ? !(e & 1) : !second) sn[e] = -sn[e];
    }
    const int partner = lane + (INTERLEAVED || !turned ? 0 : second ? -step : step);
    for (int h = h0;;) {
        const int now = h;
        Raw<F32> cur[U];
#pragma unroll
        for (int u = 0; u < U; ++u) cur[u] = raw[u];
        h += U * HPL;
        if (h < h1) load(h);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (now + u * HPL >= h1) break;
            const int hu = now + u * HPL + hl;
            const bool q = hu < a.Hq;
            float x[8];
            if constexpr (F32) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const unsigned w = cur[u].v[e >> 2][e & 3];
                    x[e] = __builtin_bit_cast(float, w);
                }
            } else {
                bf16x8(cur[u].v[0], x);
            }
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
            for (int s = 1; s < LG; s <<= 1) sum += __shfl_xor(sum, s);
            const bool normed = (q ? a.q_weight : a.k_weight) != nullptr;
            const float rs = normed ? 1.f / sqrtf(sum / (float)a.D + a.eps) : 1.f;
            float y[8], z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e] * rs * (q ? qw[e] : kw[e]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float other = INTERLEAVED ? y[e ^ 1] : __shfl(y[e], partner);
                z[e] = turned ? fmaf(y[e], c[e], other * sn[e]) : y[e];
            }
            u32x4_t o;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = __builtin_bit_cast(unsigned, bf16x2_t{(__bf16)z[2 * e], (__bf16)z[2 * e + 1]});
            if (hu < h1 && in) {
                uint16_t *to = q ? a.q_out + (size_t)m * a.qo_stride + (size_t)hu * a.D + d
                                 : a.k_out + (size_t)m * a.ko_stride + (size_t)(hu - a.Hq) * a.D + d;
                *reinterpret_cast<u32x4_t *>(to) = o;
            }
        }
        if (h >= h1) break;
    }
}

template <bool F32, bool INTERLEAVED, int LG>
void run(QkRopeArgs a, hipStream_t s) {
    constexpr int HPL = 64 / LG;
    // Waves enough for the GPU (8 a CU), each of whole loads: 32 + 8 heads of 128,
    // 64 tokens in 3.7 us, with a bound of 512 waves 4.1; 512 tokens in 5.5, with
    // 1024 6.3.  4096 bring 3 to 5% more where the rows lie in the caches (512
    // tokens 5.3) and lose 8% where they do not (1021 tokens of 36 heads of 256,
    // 10.5 us against 9.7).  Below 52 tokens all four split alike.
    const int64_t want = (2048 + a.M - 1) / a.M, loads = (a.H + HPL - 1) / HPL;
    const int64_t parts = want < loads ? want : loads;
    a.per_wave = (int)((loads + parts - 1) / parts) * HPL;
    a.parts = (a.H + a.per_wave - 1) / a.per_wave;
    const int64_t waves = (int64_t)a.M * a.parts;
    hipLaunchKernelGGL((qk_rope_kernel<F32, INTERLEAVED, LG>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, s, a);
}

template <bool F32, bool INTERLEAVED>
void pick(const QkRopeArgs &a, hipStream_t s) {
    if (a.D <= 64)
        run<F32, INTERLEAVED, 8>(a, s);
    else if (a.D <= 128)
        run<F32, INTERLEAVED, 16>(a, s);
    else if (a.D <= 256)
        run<F32, INTERLEAVED, 32>(a, s);
    else
        run<F32, INTERLEAVED, 64>(a, s);
}

}  // namespace

hipError_t launch_qk_rope(QkRopeArgs a, bool x_f32, bool interleaved, hipStream_t s) {
    if (x_f32)
        interleaved ? pick<true, true>(a, s) : pick<true, false>(a, s);
    else
        interleaved ? pick<false, true>(a, s) : pick<false, false>(a, s);
    return hipGetLastError();
}

}  // namespace qg
