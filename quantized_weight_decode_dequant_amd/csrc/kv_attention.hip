// Attention over the paged 8-bit cache for 1..32 query tokens a request (a
// decode step, or the verification of a draft, causal or as a tree).
//
//   s_t = scale * ks[page(t)] * (q . kcode_t),   p_t = softmax over visible t,
//   o = sum_t p_t vs[page(t)] vcode_t
//
// The query heads that share a KV head and the query tokens of a request
// are rows of one product: row = token * G + head, 16 rows to a tile.  A wave
// takes steps of 32 tokens.  S^T = K Q^T on the 16x16x32 f16 MFMA (codes are
// exact in f16; q is scaled by a power of two per row into f16's range), so
// lane (g, c) holds the scores of row c for the tokens 4g.. of each 16, and
// these are the tokens whose values its V load brings: O^T += V^T P^T takes
// the probabilities from their registers.  Sums, maxima and O are fp32; p is
// rounded to f16 (11 bits; the output has 8 in bf16).  The running maximum
// is only raised when a score passes it by 8 (in powers of two: p <= 2^8 is
// far inside f16), so most steps neither exchange across lanes nor rescale O.
// The value scales enter p as vs / vref with vref a power of two at least as
// large as every vs so far, wave-uniform.
//
// A workgroup takes one chunk of a request's tokens for one KV head and up to
// 16 * NR * RS rows; its waves split the chunk's steps (TS of them) and the
// rows (RS) and join in LDS.  Several chunks are joined by a second kernel.
#include "kv_cache.h"

namespace qg {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr int AT_WAVES = 4;
constexpr float NEG_INF = -__builtin_inff();

// 8 codes (two words) as the f16 operand
template <bool E4M3>
__device__ __forceinline__ f16x8_t codes8(unsigned w0, unsigned w1) {
    f16x2_t p[4];
    if (E4M3) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, true);
    } else {
        // byte b ^ 0x80 under the f16 exponent of 1024: 1024 + 128 + code
        w0 ^= 0x80808080u;
        w1 ^= 0x80808080u;
        const f16x2_t bias = {(_Float16)1152.f, (_Float16)1152.f};
        p[0] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, w0, 0x04010400u)) - bias;
        p[1] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, w0, 0x04030402u)) - bias;
        p[2] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, w1, 0x04010400u)) - bias;
        p[3] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, w1, 0x04030402u)) - bias;
    }
    return f16x8_t{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

__device__ __forceinline__ float readlane_f(float v, int l) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}

// the smallest power of two >= x (x > 0)
__device__ __forceinline__ float pow2_above(float x) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    return __builtin_bit_cast(float, (u + 0x7FFFFFu) & 0x7F800000u);
}

// tokens [first, end) that some row of the request may see, and the chunks
// that hold them
struct Span {
    int len, T, first, c0, c1;
    bool too_long;  // longer than the call was told of: its rows become NaN
};

__device__ __forceinline__ Span span_of(const KvAttnArgs &a, int r) {
    Span s;
    const int q0 = a.q_start[r];
    s.T = min(max(a.q_start[r + 1] - q0, 0), a.max_q);
    if (q0 < 0 || q0 + s.T > a.M) s.T = 0;
    s.len = min(max(a.lens[r], 0), a.max_blocks * a.page);
    s.first = a.window > 0 ? max(s.len - s.T - a.window + 1, 0) : 0;
    s.c0 = s.first / a.chunk;
    s.c1 = (s.len + a.chunk - 1) / a.chunk;
    s.too_long = s.c1 - s.c0 > a.chunks;
    return s;
}

}  // namespace

template <bool E4M3, int D, int NR, int RS>
__global__ void __launch_bounds__(AT_WAVES * 64) kv_attn_kernel(KvAttnArgs a) {
    constexpr int TS = AT_WAVES / RS;   // waves that split the tokens
    constexpr int KS = D / 32;          // MFMA steps of Q K^T
    constexpr int DT = D / 16;          // tiles of O
    __shared__ float slots[TS > 1 ? 2 * RS : 1][TS > 1 ? NR * (DT * 4 + 2) : 1][64];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c = lane & 15;
    const int ts = wave / RS, rsi = wave % RS;
    const int bx = blockIdx.x;
    const int ci = bx % a.chunks, rh = bx / a.chunks;
    const int r = rh / a.Hkv, h = rh % a.Hkv;
    const Span sp = span_of(a, r);
    const int rows = sp.T * a.G;
    const int row0 = blockIdx.y * (16 * NR * RS);
    if (row0 >= rows) return;
    const int chunk = sp.c0 + ci;
    if (chunk >= sp.c1 && !(ci == 0 && sp.c0 >= sp.c1)) return;  // chunk 0 of an empty request writes zeros
    const int q0 = a.q_start[r];
    const int base = sp.len - sp.T;  // position of the first query token

    // Q, as f16 in the K tiles' order of dimensions
    f16x8_t qf[NR][KS];
    float cs[NR];    // softmax scale and q's power of two
    int rowm[NR], rowh[NR], pos[NR];
    unsigned tree[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int row = row0 + 16 * (rsi * NR + n) + c;
        const bool valid = row < rows;
        const int j = valid ? row / a.G : 0;
        rowm[n] = valid ? q0 + j : -1;
        rowh[n] = h * a.G + (valid ? row % a.G : 0);
        pos[n] = base + j;
        tree[n] = a.tree && valid ? a.tree[q0 + j] : 0u;
        const uint16_t *q = a.q + (size_t)(q0 + j) * a.q_stride + (size_t)rowh[n] * D;
        float v[KS][8];
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const u32x4_t w = *reinterpret_cast<const u32x4_t *>(q + 64 * (s >> 1) + 16 * g + 8 * (s & 1));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[s][2 * e] = bf16_lo(w[e]);
                v[s][2 * e + 1] = bf16_hi(w[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[s][e]));
        }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        // the row's largest magnitude to [2^13, 2^14)
        const int e2 = top > 0.f ? 13 - ((int)(__builtin_bit_cast(unsigned, top) >> 23) - 127) : 0;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) qf[n][s][e] = (_Float16)ldexpf(v[s][e], e2);
        cs[n] = ldexpf(a.scale, -e2);
    }

    f32x4_t o[NR][DT];
    float m[NR], l[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        m[n] = NEG_INF;
        l[n] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    float vref = 0.f;

    const int t_lo = max(chunk * a.chunk, sp.first & ~(KV_STEP - 1));
    const int t_hi = min((chunk + 1) * a.chunk, sp.len);
    // the chunk's pages and their scales, one a lane
    const int page0 = t_lo / a.page;
    int my_page = -1;
    float my_ks = 0.f, my_vs = 0.f;
    if (page0 + lane < a.max_blocks && (page0 + lane) * a.page < t_hi) {
        my_page = a.table[(size_t)r * a.max_blocks + page0 + lane];
        if (my_page < 0 || my_page >= a.pages) my_page = -1;
        if (my_page >= 0) {
            my_ks = a.k_scales[(size_t)my_page * a.Hkv + h];
            my_vs = a.v_scales[(size_t)my_page * a.Hkv + h];
        }
    }
    for (int t0 = t_lo + ts * KV_STEP; t0 < t_hi; t0 += TS * KV_STEP) {
        const int pi = t0 / a.page - page0;
        const int page = __builtin_amdgcn_readlane(my_page, pi);
        if (page < 0) continue;  // a page that is not there is not attended to
        const float ks = readlane_f(my_ks, pi), vs = readlane_f(my_vs, pi);
        const int in = t0 % a.page;
        const size_t block = ((size_t)page * a.Hkv + h) * ((size_t)a.page * D) + (size_t)in * D;
        const u32x4_t *kp = reinterpret_cast<const u32x4_t *>(a.k + block) + lane;
        const u32x4_t *vp = reinterpret_cast<const u32x4_t *>(a.v + block) + lane;
        u32x4_t kw[2][D / 64], vw[D / 32];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int u = 0; u < D / 64; ++u) kw[i][u] = kp[(i * (D / 64) + u) * 64];
#pragma unroll
        for (int u = 0; u < D / 32; ++u) vw[u] = vp[u * 64];

        // scores
        f32x4_t s[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) s[n][0] = s[n][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const u32x4_t w = kw[i][k >> 1];
                const f16x8_t kf = codes8<E4M3>(w[2 * (k & 1)], w[2 * (k & 1) + 1]);
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    s[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[n][k], s[n][i], 0, 0, 0);
            }
        // the value scale: O is in units of vref
        float ratio = 0.f;
        if (vs > 0.f) {
            if (vs > vref) {
                const float up = pow2_above(vs), f = vref / up;
                vref = up;
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[n][d] *= f;
            }
            ratio = vs / vref;
        }
        const bool mask = t0 + KV_STEP - 1 > base || t0 < sp.len - a.window * (a.window > 0);
        f16x8_t pf[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float f = ks * cs[n];
            float x[8];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * i + e] = s[n][i][e] * f;
            if (mask) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int t = t0 + 16 * (e >> 2) + 4 * g + (e & 3);
                    bool see = t < sp.len;
                    if (a.tree)
                        see = see && (t < base || ((tree[n] >> ((t - base) & 31)) & 1u));
                    else
                        see = see && t <= pos[n] && (a.window <= 0 || t > pos[n] - a.window);
                    x[e] = see ? x[e] : NEG_INF;
                }
            }
            float top = x[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
            if (__any(top > m[n] + 8.f)) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                // only the rows concerned: a row does not depend on its neighbours
                const float mn = top > m[n] + 8.f ? top : m[n];
                const float down = mn == NEG_INF ? 1.f : __builtin_amdgcn_exp2f(m[n] - mn);
                m[n] = mn;
                l[n] *= down;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[n][d] *= down;
            }
            const float ref = m[n] == NEG_INF ? 0.f : m[n];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = __builtin_amdgcn_exp2f(x[e] - ref);
                l[n] += p;
                pf[n][e] = (_Float16)(p * ratio);
            }
        }
        // codes of slots behind the last token may be anything (an E4M3 NaN)
        if (t0 + KV_STEP > sp.len) {
            unsigned keep[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t0 + 16 * i + 4 * g + e < sp.len) keep[i] |= 0xFFu << (8 * e);
#pragma unroll
            for (int u = 0; u < D / 32; ++u) {
                vw[u][0] &= keep[0];
                vw[u][1] &= keep[1];
                vw[u][2] &= keep[0];
                vw[u][3] &= keep[1];
            }
        }
#pragma unroll
        for (int u = 0; u < D / 32; ++u)
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const f16x8_t vf = codes8<E4M3>(vw[u][2 * d], vw[u][2 * d + 1]);
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    o[n][2 * u + d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[n], o[n][2 * u + d], 0, 0, 0);
            }
    }
    // in true units, each wave its own maximum; the sum over the lanes' tokens
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        l[n] += __shfl_xor(l[n], 16);
        l[n] += __shfl_xor(l[n], 32);
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] *= vref;
    }
    // join the waves that split the tokens, half of them at a time
    if constexpr (TS > 1) {
#pragma unroll
        for (int half = TS / 2; half; half >>= 1) {
            __syncthreads();
            if (ts >= half && ts < 2 * half) {
                float(*to)[64] = slots[(ts - half) * RS + rsi];
#pragma unroll
                for (int n = 0; n < NR; ++n) {
#pragma unroll
                    for (int d = 0; d < DT; ++d)
#pragma unroll
                        for (int e = 0; e < 4; ++e) to[n * (DT * 4 + 2) + 4 * d + e][lane] = o[n][d][e];
                    to[n * (DT * 4 + 2) + DT * 4][lane] = m[n];
                    to[n * (DT * 4 + 2) + DT * 4 + 1][lane] = l[n];
                }
            }
            __syncthreads();
            if (ts < half) {
                float(*from)[64] = slots[ts * RS + rsi];
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    const float m2 = from[n * (DT * 4 + 2) + DT * 4][lane];
                    const float l2 = from[n * (DT * 4 + 2) + DT * 4 + 1][lane];
                    const float mn = fmaxf(m[n], m2);
                    const float f1 = mn == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(m[n] - mn);
                    const float f2 = mn == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(m2 - mn);
                    m[n] = mn;
                    l[n] = l[n] * f1 + l2 * f2;
#pragma unroll
                    for (int d = 0; d < DT; ++d)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[n][d][e] = o[n][d][e] * f1 + from[n * (DT * 4 + 2) + 4 * d + e][lane] * f2;
                }
            }
        }
    }
    if (ts != 0) return;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        if (rowm[n] < 0) continue;
        if (a.chunks == 1) {
            const float f = sp.too_long ? __builtin_nanf("") : l[n] == 0.f ? 0.f : 1.f / l[n];
            const size_t at = (size_t)rowm[n] * a.out_stride + (size_t)rowh[n] * D + 4 * g;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const f32x4_t v = o[n][d] * f;
                if (a.out_f32)
                    *reinterpret_cast<f32x4_t *>((float *)a.out + at + 16 * d) = v;
                else
                    *reinterpret_cast<u32x2_t *>((uint16_t *)a.out + at + 16 * d) =
                        u32x2_t{(unsigned)f32_to_bf16(v[0]) | ((unsigned)f32_to_bf16(v[1]) << 16),
                                (unsigned)f32_to_bf16(v[2]) | ((unsigned)f32_to_bf16(v[3]) << 16)};
            }
        } else {
            const size_t at = ((size_t)ci * a.M + rowm[n]) * a.Hq + rowh[n];
#pragma unroll
            for (int d = 0; d < DT; ++d)
                *reinterpret_cast<f32x4_t *>(a.part + at * D + 16 * d + 4 * g) = o[n][d];
            if (g == 0) *reinterpret_cast<f32x2_t *>(a.part_ml + 2 * at) = f32x2_t{m[n], l[n]};
        }
    }
}

// Joins the chunks of one (query token, head): one wave, D / 64 dimensions a lane.
template <int D>
__global__ void __launch_bounds__(64) kv_attn_join_kernel(KvAttnArgs a) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x;
    const int r = blockIdx.x / a.max_q, j = blockIdx.x % a.max_q, hq = blockIdx.y;
    const Span sp = span_of(a, r);
    if (j >= sp.T) return;
    const int row = a.q_start[r] + j;
    const int n = max(min(sp.c1 - sp.c0, a.chunks), 1);
    const size_t at = (size_t)row * a.Hq + hq, step = (size_t)a.M * a.Hq;
    float mx = NEG_INF;
    for (int c = lane; c < n; c += 64) mx = fmaxf(mx, a.part_ml[2 * (at + c * step)]);
#pragma unroll
    for (int d = 32; d; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
    float o[E], l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int c = 0; c < n; ++c) {
        // (a row of NaN scores has no maximum, but a NaN sum)
        const float f = mx == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(a.part_ml[2 * (at + c * step)] - mx);
        l += f * a.part_ml[2 * (at + c * step) + 1];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += f * a.part[(at + c * step) * D + e * 64 + lane];
    }
    const float f = sp.too_long ? __builtin_nanf("") : l == 0.f ? 0.f : 1.f / l;
    const size_t to = (size_t)row * a.out_stride + (size_t)hq * D + lane;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (a.out_f32)
            ((float *)a.out)[to + 64 * e] = o[e] * f;
        else
            ((uint16_t *)a.out)[to + 64 * e] = f32_to_bf16(o[e] * f);
    }
}

void kv_attention_split(int64_t R, int64_t Hkv, int64_t rows, int64_t page, int64_t span,
                        bool windowed, int *chunk, int64_t *chunks) {
    const int64_t groups = (R > 0 ? R : 1) * Hkv * ((rows + 127) / 128);
    // about four workgroups to a CU
    const int64_t want = (1024 + groups - 1) / groups;
    int64_t c = (span + want - 1) / want;
    if (c < 128) c = 128;
    if (c > KV_CHUNK_MAX) c = KV_CHUNK_MAX;
    const int64_t unit = page > 128 ? page : 128;
    c = (c + unit - 1) / unit * unit;
    *chunk = (int)c;
    // a window need not start where a chunk does
    *chunks = (span + c - 1) / c + (windowed ? 1 : 0);
}

namespace {

template <bool E4M3, int D, int NR, int RS>
void run(const KvAttnArgs &a, hipStream_t s) {
    const int rows = a.max_q * a.G;
    const dim3 grid((unsigned)(a.R * a.Hkv * a.chunks), (unsigned)((rows + 16 * NR * RS - 1) / (16 * NR * RS)));
    hipLaunchKernelGGL((kv_attn_kernel<E4M3, D, NR, RS>), grid, dim3(AT_WAVES * 64), 0, s, a);
    if (a.chunks > 1)
        hipLaunchKernelGGL((kv_attn_join_kernel<D>), dim3((unsigned)(a.R * a.max_q), (unsigned)a.Hq), dim3(64), 0, s, a);
}

template <bool E4M3, int D>
void pick(const KvAttnArgs &a, hipStream_t s) {
    const int rows = a.max_q * a.G;
    if (rows <= 16)
        run<E4M3, D, 1, 1>(a, s);
    else if (rows <= 32)
        run<E4M3, D, 1, 2>(a, s);
    else
        run<E4M3, D, 1, 4>(a, s);
}

}  // namespace

hipError_t launch_kv_attention(const KvAttnArgs &a, int D, bool e4m3, hipStream_t s) {
    if (e4m3)
        D == 64 ? pick<true, 64>(a, s) : D == 128 ? pick<true, 128>(a, s) : pick<true, 256>(a, s);
    else
        D == 64 ? pick<false, 64>(a, s) : D == 128 ? pick<false, 128>(a, s) : pick<false, 256>(a, s);
    return hipGetLastError();
}

}  // namespace qg
