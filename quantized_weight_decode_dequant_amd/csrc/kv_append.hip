// New keys and values written into the paged 8-bit cache.
//
// Per page and head: s = max(s_old, amax * (1 / top)) with amax over the new
// tokens' finite values, 1 / top the fp32 nearest to 1/127 (int8) or 1/448
// (E4M3) and s_old = 0 where the first of the new tokens opens the page; inv = 1 / s; code = round(x *
// inv), clamped to +-top.  Where s grew, the page's codes are rounded again
// from code * (s_old / s).  Each of these steps is one correctly rounded
// fp32 operation (round to nearest even), so the codes do not depend on how
// the work is split.
//
// One workgroup per (run of slots that lie in one page, head, K or V): the
// largest magnitude first, then, with the values read again from the caches,
// the codes.  Latency bounds a few tokens: slot, run, values, scale in turn,
// 5.2 us for 64 single ones (8 heads of 128, pages of 64) where no scale grows;
// then a page's codes, read and written back one 16-byte piece a lane after the
// other: 8.3 us where 6% of the blocks grow, as they do for tokens that are
// alike, 9.5 where all do (heads of 256, pages of 256: 8, 21 and 33 us).  The
// two passes bound many tokens (11460 of 7 prompts: 21 us, 3.4 TB/s).  Keys: a
// thread codes 16 dimensions of a token, one 16-byte piece of the block, with
// the tokens along the lanes, so that a wave writes whole kilobytes.  Values,
// which the block holds by token within a dimension: a thread codes 2 x 2
// dimensions of 8 tokens, two whole 16-byte pieces; where some of the 8 tokens
// are not the run's, byte by byte.
#include <type_traits>

#include "kv_cache.h"

namespace qg {

namespace {

constexpr float AP_TINY = 0x1p-100f;  // blocks below this are stored as zeros

// The codes of four values x * inv.  FINITE: all of the run's values are, so
// |x * inv| exceeds the largest code by rounding only and neither a clamp nor
// a test for NaN is needed; an int8 code is then the low byte of the sum with
// 1.5 * 2^23, which rounds to nearest even.  Otherwise infinities become the
// largest code and NaN 0.
template <bool E4M3, bool FINITE>
__device__ __forceinline__ unsigned encode4(float a, float b, float c, float d, float inv) {
#pragma clang fp contract(off)  // the product is rounded before it is coded
    float z[4] = {a * inv, b * inv, c * inv, d * inv};
    if (!FINITE) {
        constexpr float top = E4M3 ? 448.f : 127.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = z[i] == z[i] ? fminf(fmaxf(z[i], -top), top) : 0.f;
    }
    if (E4M3) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
        return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], lo, true);
    }
    unsigned u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __builtin_bit_cast(unsigned, z[i] + 12582912.f);
    const unsigned lo = __builtin_amdgcn_perm(u[1], u[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(u[3], u[2], 0x04000C0Cu);
    return lo | hi;
}

template <bool E4M3, int B>
__device__ __forceinline__ float decode(unsigned w) {
    if (E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)w, B);
    return (float)(int8_t)((w >> (8 * B)) & 0xFFu);
}

// larger halves of two pairs of bf16 magnitudes, as bits (which order like them)
__device__ __forceinline__ unsigned max_pair(unsigned a, unsigned b) {
    typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}

// the same bits where the bf16 is finite, else 0
__device__ __forceinline__ unsigned finite_pair(unsigned w) {
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
    return w;
}

constexpr unsigned MAGNITUDE = 0x7FFF7FFFu;

}  // namespace

template <bool E4M3, int T>
__global__ void __launch_bounds__(T) kv_append_kernel(KvAppendArgs a) {
    __shared__ unsigned wmax[T / 64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int h = blockIdx.y;
    const bool value = blockIdx.z != 0;
    const int64_t stride = value ? a.v_stride : a.k_stride;
    const int D = a.D, page = a.page;
    const uint16_t *X = (value ? a.V : a.K) + (size_t)h * D;
    constexpr float inv_top = E4M3 ? 1.f / 448.f : 1.f / 127.f;

    // the tokens of this workgroup's chunk that start a run
    const int m0 = blockIdx.x * a.chunk;
    int my_slot = -1;
    bool starts = false;
    if (lane < a.chunk && m0 + lane < a.M) {
        my_slot = a.slots[m0 + lane];
        starts = my_slot >= 0 && my_slot < a.slots_end &&
                 (my_slot % page == 0 || m0 + lane == 0 || a.slots[m0 + lane - 1] != my_slot - 1);
    }
    for (unsigned long long left = __ballot(starts); left; left &= left - 1) {
        const int i = __builtin_ctzll(left), m = m0 + i;
        const int slot = __builtin_amdgcn_readlane(my_slot, i), off = slot % page;
        const size_t block = (size_t)(slot / page) * a.Hkv + h;
        uint8_t *codes = (value ? a.v : a.k) + block * page * D;
        float *scale = (value ? a.v_scales : a.k_scales) + block;
        const float s_old = off ? *scale : 0.f;
        const uint16_t *x = X + (size_t)m * stride;
        // its length (every wave finds it by itself)
        int n = min(page - off, a.M - m);
        for (int k = 0; k < n; k += 64) {
            const bool breaks = k + lane < n && a.slots[m + k + lane] != slot + k + lane;
            const unsigned long long b = __ballot(breaks);
            if (b) n = k + __builtin_ctzll(b);
        }
        // the largest magnitude's bits; a second time without what is not
        // finite, if that is the largest
        const int per = D >> 3;  // 16-byte pieces of a token
        bool finite = true;
        unsigned top;
        for (;;) {
            unsigned pair = 0u;
#pragma unroll 4
            for (int e = tid; e < n * per; e += T) {
                const int t = (unsigned)e / (unsigned)per;
                const u32x4_t w = *reinterpret_cast<const u32x4_t *>(x + (size_t)t * stride + 8 * (e - t * per));
#pragma unroll
                for (int j = 0; j < 4; ++j) pair = max_pair(pair, finite ? w[j] & MAGNITUDE : finite_pair(w[j]) & MAGNITUDE);
            }
            top = max(pair & 0xFFFFu, pair >> 16);
#pragma unroll
            for (int d = 32; d; d >>= 1) top = max(top, __shfl_xor(top, d));
            if (T > 64) {
                if (lane == 0) wmax[tid >> 6] = top;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < T / 64; ++w) top = max(top, wmax[w]);
                __syncthreads();
            }
            if (top < 0x7F80u) break;
            finite = false;
        }
        float amax = __builtin_bit_cast(float, top << 16);
        if (amax < AP_TINY) amax = 0.f;
        const float s = fmaxf(s_old, amax * inv_top);
        const float inv = s > 0.f ? 1.f / s : 0.f;
        if (off && s > s_old) {
            const float ratio = s_old / s;
            u32x4_t *p = reinterpret_cast<u32x4_t *>(codes);
            for (int e = tid; e < page * D / 16; e += T) {
                u32x4_t w = p[e];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = encode4<E4M3, true>(decode<E4M3, 0>(w[j]), decode<E4M3, 1>(w[j]),
                                               decode<E4M3, 2>(w[j]), decode<E4M3, 3>(w[j]), ratio);
                p[e] = w;
            }
        }
        __syncthreads();  // every thread has read the scale and its old codes are written
        if (tid == 0) *scale = s;
        const auto put = [&](auto all_finite) {
            const auto code = [&](float p, float q, float r, float u) {
                return encode4<E4M3, decltype(all_finite)::value>(p, q, r, u, inv);
            };
            if (!value) {
                // 16 tokens along the lanes, then the 16-dimension pieces, from the
                // 16-token tile on that holds the run's first token
                const int t_first = off & ~15, tiles = ((off + n - 1) >> 4) - (off >> 4) + 1, pieces = D >> 4;
#pragma unroll 2
                for (int e = tid; e < tiles * 16 * pieces; e += T) {
                    const int q = e >> 4, tile = (unsigned)q / (unsigned)pieces, piece = q - tile * pieces;
                    const int t = t_first + tile * 16 + (e & 15);
                    if (t < off || t >= off + n) continue;
                    const u32x4_t *p = reinterpret_cast<const u32x4_t *>(x + (size_t)(t - off) * stride + 16 * piece);
                    const u32x4_t w[2] = {p[0], p[1]};
                    u32x4_t o;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const unsigned lo = w[j >> 1][2 * (j & 1)], hi = w[j >> 1][2 * (j & 1) + 1];
                        o[j] = code(bf16_lo(lo), bf16_hi(lo), bf16_lo(hi), bf16_hi(hi));
                    }
                    *reinterpret_cast<u32x4_t *>(codes + (t >> 4) * 16 * D + piece * 256 + (t & 15) * 16) = o;
                }
            } else {
                // 8 pairs of dimensions along the lanes, then the four token
                // groups, then the 32-dimension columns
                const int t_first = off & ~31, tiles = ((off + n - 1) >> 5) - (off >> 5) + 1, cols = D >> 5;
                for (int e = tid; e < tiles * cols * 32; e += T) {
                    const int q = e >> 5, tile = (unsigned)q / (unsigned)cols, col = q - tile * cols;
                    const int g = (e >> 3) & 3, d = 32 * col + 2 * (e & 7), t0 = t_first + 32 * tile + 4 * g;
                    uint8_t *to = codes + (t0 >> 5) * 32 * D + col * 1024 + g * 256 + 2 * (e & 7) * 16;
                    if (t0 >= off && t0 + 20 <= off + n) {
                        u32x4_t o[2];
#pragma unroll
                        for (int dh = 0; dh < 2; ++dh)
#pragma unroll
                            for (int th = 0; th < 2; ++th) {
                                unsigned w[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    w[k] = *reinterpret_cast<const unsigned *>(x + (size_t)(t0 + 16 * th + k - off) * stride + d + 16 * dh);
                                o[0][2 * dh + th] = code(bf16_lo(w[0]), bf16_lo(w[1]), bf16_lo(w[2]), bf16_lo(w[3]));
                                o[1][2 * dh + th] = code(bf16_hi(w[0]), bf16_hi(w[1]), bf16_hi(w[2]), bf16_hi(w[3]));
                            }
                        reinterpret_cast<u32x4_t *>(to)[0] = o[0];
                        reinterpret_cast<u32x4_t *>(to)[1] = o[1];
                    } else {
                        for (int k = 0; k < 8; ++k) {
                            const int t = t0 + 16 * (k >> 2) + (k & 3);
                            if (t < off || t >= off + n) continue;
#pragma unroll
                            for (int dh = 0; dh < 2; ++dh) {
                                const unsigned w = *reinterpret_cast<const unsigned *>(x + (size_t)(t - off) * stride + d + 16 * dh);
                                const unsigned o = code(bf16_lo(w), bf16_hi(w), 0.f, 0.f);
                                to[8 * dh + k] = (uint8_t)o;
                                to[16 + 8 * dh + k] = (uint8_t)(o >> 8);
                            }
                        }
                    }
                }
            }
        };
        if (finite)
            put(std::true_type());
        else
            put(std::false_type());
    }
}

namespace {

template <int T>
void run(const KvAppendArgs &a, bool e4m3, hipStream_t s) {
    const dim3 grid((unsigned)((a.M + a.chunk - 1) / a.chunk), (unsigned)a.Hkv, 2);
    if (e4m3)
        hipLaunchKernelGGL((kv_append_kernel<true, T>), grid, dim3(T), 0, s, a);
    else
        hipLaunchKernelGGL((kv_append_kernel<false, T>), grid, dim3(T), 0, s, a);
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs &args, bool e4m3, hipStream_t s) {
    KvAppendArgs a = args;
    // Few tokens: a wave for each token that may start a run.  Many (prompts,
    // whose runs are pages): a workgroup of four waves for each 32 tokens, the
    // shortest page, which takes the runs that start there in turn.  What the
    // runs are stands in `slots`, on the GPU, so M decides alone.  Measured
    // (int8, 8 heads of 128, pages of 64; waves against workgroups): single
    // tokens, 64 of them 5.2 us against 58, 1024 18 against 64, 1025 19 against
    // 68, 4096 58 against 133; drafts of 16 tokens, 16 of them 14.3 against
    // 12.6, 64 47 against 14, 65 48 against 14; one prompt of 300 tokens 10.4
    // against 6.0, of 1000 16 against 6.6, of 11460 84 against 20 (pages of 128).
    // So the rule fits single tokens up to 1024 and prompts above; drafts and
    // prompts of up to 1024 tokens take up to 5 times what the other variant
    // would (a prompt of 1024 on pages and heads of 256: 112 against 23), more
    // single tokens than 1024 up to 3.6 times.
    if (a.M <= 1024) {
        a.chunk = 1;
        run<64>(a, e4m3, s);
    } else {
        a.chunk = 32;
        run<256>(a, e4m3, s);
    }
    return hipGetLastError();
}

}  // namespace qg
