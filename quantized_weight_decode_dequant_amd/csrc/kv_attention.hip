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
// large as every vs of the chunk.
//
// A workgroup takes one chunk of a request's tokens for one KV head and up to
// 16 * NR * RS rows; its waves split the chunk's steps (TS of them) and the
// rows (RS) and join in LDS.  Several chunks are joined by a second kernel.
#include "kv_cache.h"

namespace qg {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr float NEG_INF = -__builtin_inff();

// An int8 code c enters the MFMA as the f16 whose bits are c + 128: a
// denormal (which the MFMA keeps), worth (c + 128) 2^-24.  The products'
// accumulators are corrected by -128 times the other operand's sum.
template <bool E4M3>
struct Code {
    static constexpr float unit = E4M3 ? 1.f : 0x1p24f;
    static constexpr float bias = E4M3 ? 0.f : 128.f;
};

// 8 codes (two words) as the f16 operand
template <bool E4M3>
__device__ __forceinline__ f16x8_t codes8(unsigned w0, unsigned w1) {
    u32x4_t o;
    if (E4M3) {
        o[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, false));
        o[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, true));
        o[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, false));
        o[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, true));
    } else {
        w0 ^= 0x80808080u;
        w1 ^= 0x80808080u;
        o[0] = __builtin_amdgcn_perm(0u, w0, 0x0C010C00u);  // selector 0x0C: a zero byte
        o[1] = __builtin_amdgcn_perm(0u, w0, 0x0C030C02u);
        o[2] = __builtin_amdgcn_perm(0u, w1, 0x0C010C00u);
        o[3] = __builtin_amdgcn_perm(0u, w1, 0x0C030C02u);
    }
    return __builtin_bit_cast(f16x8_t, o);
}

__device__ __forceinline__ float readlane_f(float v, int l) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}

// four values rounded to bf16 (to nearest even)
__device__ __forceinline__ u32x2_t bf16x4(f32x4_t v) {
    return u32x2_t{__builtin_bit_cast(unsigned, bf16x2_t{(__bf16)v[0], (__bf16)v[1]}),
                   __builtin_bit_cast(unsigned, bf16x2_t{(__bf16)v[2], (__bf16)v[3]})};
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

// One wave's loads of N kilobytes, 128 bits a lane, through a buffer resource
// over the page's block: `bytes` of 0 reads nothing and gives zeros, so the
// loads are issued on every path and a wait for earlier ones leaves them in
// flight.
template <int N, bool NT>
__device__ __forceinline__ void load_codes(u32x4_t (&to)[N], const uint8_t *block, unsigned bytes, unsigned at, int lane) {
    const __amdgpu_buffer_rsrc_t r = make_rsrc(block, bytes);
#pragma unroll
    for (int u = 0; u < N; ++u)
        to[u] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                r, 16 * lane + u % 4 * 1024, (int)at + u / 4 * 4096, NT ? 2 : 0));
}

template <bool E4M3, int D, int NR, int RS, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, 2) kv_attn_kernel(KvAttnArgs a) {
    constexpr int TS = WAVES / RS;      // waves that split the tokens
    constexpr int KS = D / 32;          // MFMA steps of Q K^T
    constexpr int DT = D / 16;          // tiles of O
    constexpr int SL = DT * 4 + 2;      // floats a lane and row tile joins
    constexpr float UNIT = Code<E4M3>::unit, BIAS = Code<E4M3>::bias;
    constexpr bool NT = RS == 1;        // read by one wave only: past the caches
    __shared__ float slots[TS > 1 ? (TS / 2) * RS : 1][TS > 1 ? NR * SL : 1][64];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c = lane & 15;
    const int ts = wave / RS, rsi = wave % RS;
    // chunk index slowest: workgroups go to the XCDs in turn, and most late
    // chunks are empty where lengths differ
    const int nrh = a.R * a.Hkv;
    const int ci = blockIdx.x / nrh, rh = blockIdx.x % nrh;
    const int r = rh / a.Hkv, h = rh % a.Hkv;
    const Span sp = span_of(a, r);
    const int rows = sp.T * a.G;
    const int row0 = blockIdx.y * (16 * NR * RS);
    if (row0 >= rows) return;
    const int chunk = sp.c0 + ci;
    if (chunk >= sp.c1 && !(ci == 0 && sp.c0 >= sp.c1)) return;  // chunk 0 of an empty request writes zeros
    const int q0 = a.q_start[r];
    const int base = sp.len - sp.T;  // position of the first query token

    // the chunk's pages and their scales, one a lane
    const int t_lo = max(chunk * a.chunk, sp.first & ~(KV_STEP - 1));
    const int t_hi = min((chunk + 1) * a.chunk, sp.len);
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
    // vref: a power of two at least as large as every value scale of the chunk
    float vref = fmaxf(my_vs, 0.f);
#pragma unroll
    for (int d = 32; d; d >>= 1) vref = fmaxf(vref, __shfl_xor(vref, d));
    vref = readlane_f(vref > 0.f ? pow2_above(vref) : 1.f, 0);
    // the page's value scale over vref, as a power of two in the exponent, and
    // its inverse (a page whose values are all 0: no scale)
    const bool my_v = my_vs > 0.f;
    const float my_lr = my_v ? __builtin_amdgcn_logf(my_vs / vref) : 0.f, my_rr = my_v ? vref / my_vs : 1.f;
    const int shift = __builtin_ctz(a.page);
    // the loads of the step at t (past the end, or of a page that is not
    // there: none)
    u32x4_t kw[D / 32], vw[D / 32];
    const auto page_at = [&](int t) { return t < t_hi ? __builtin_amdgcn_readlane(my_page, (t >> shift) - page0) : -1; };
    const auto load = [&](u32x4_t(&to)[D / 32], const uint8_t *codes, int t) {
        const int page = page_at(t);
        const size_t at = ((size_t)max(page, 0) * a.Hkv + h) * ((size_t)a.page * D);
        load_codes<D / 32, NT>(to, uniform_ptr(codes + at), page < 0 ? 0u : (unsigned)a.page * D,
                               (unsigned)(t & (a.page - 1)) * D, lane);
    };
    const int first = t_lo + ts * KV_STEP;
    load(kw, a.k, first);
    load(vw, a.v, first);

    // Q, as f16 in the K tiles' order of dimensions
    f16x8_t qf[NR][KS];
    float cs[NR], k0[NR];  // factor and start of the scores
    int rowm[NR], rowh[NR], pos[NR], lo[NR];  // visible: lo < t <= pos
    unsigned tree[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int row = row0 + 16 * (rsi * NR + n) + c;
        const bool valid = row < rows;
        const int j = valid ? row / a.G : 0;
        rowm[n] = valid ? q0 + j : -1;
        rowh[n] = h * a.G + (valid ? row % a.G : 0);
        pos[n] = base + j;
        lo[n] = a.window > 0 ? pos[n] - a.window : -1;
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
        // the row's largest magnitude to [2^13, 2^14), the scale's sign with it
        const int e2 = top > 0.f ? 13 - ((int)(__builtin_bit_cast(unsigned, top) >> 23) - 127) : 0;
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = ldexpf(v[s][e], e2);
                const _Float16 hx = (_Float16)(a.scale < 0.f ? -x : x);
                qf[n][s][e] = hx;
                sum += (float)hx;
            }
        if (BIAS != 0.f) {
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
        }
        k0[n] = -(BIAS / UNIT) * sum;
        cs[n] = ldexpf(fabsf(a.scale) * UNIT, -e2);
    }

    f32x4_t o[NR][DT];  // sums of p times values, in units of vref (/ UNIT, biased)
    float m[NR], nm[NR], l[NR], ps[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        m[n] = NEG_INF;
        nm[n] = l[n] = ps[n] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    const f16x8_t ones = {(_Float16)1.f, (_Float16)1.f, (_Float16)1.f, (_Float16)1.f,
                          (_Float16)1.f, (_Float16)1.f, (_Float16)1.f, (_Float16)1.f};

    // A step's keys are replaced by the next step's once they are used, then
    // its values: one buffer each, with loads in flight all the time.
    constexpr int STRIDE = TS * KV_STEP;
    for (int t0 = first; t0 < t_hi; t0 += STRIDE) {
        // a page that is not there is not attended to
        const bool there = page_at(t0) >= 0;
        const int pi = (t0 >> shift) - page0;
        const float ks = readlane_f(my_ks, pi), lr = readlane_f(my_lr, pi), rr = readlane_f(my_rr, pi);
        const bool no_v = !(readlane_f(my_vs, pi) > 0.f);
        // scores
        f32x4_t s[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) s[n][0] = s[n][1] = f32x4_t{k0[n], k0[n], k0[n], k0[n]};
        // (the barriers keep the compiler from converting every code first,
        // which takes more registers than there are)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const u32x4_t w = kw[i * (D / 64) + (k >> 1)];
                const f16x8_t kf = codes8<E4M3>(w[2 * (k & 1)], w[2 * (k & 1) + 1]);
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    s[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[n][k], s[n][i], 0, 0, 0);
            }
            if (k & 1) __builtin_amdgcn_sched_barrier(0);
        }
        load(kw, a.k, t0 + STRIDE);
        // codes of slots behind the last token may be anything (an E4M3 NaN),
        // and those of a page without a value scale are worth nothing
        if (t0 + KV_STEP > sp.len || no_v) {
            unsigned keep[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) keep[i] |= (t0 + 16 * i + 4 * g + e < sp.len) & !no_v ? 0xFFu << (8 * e) : 0u;
#pragma unroll
            for (int u = 0; u < D / 32; ++u) {
                vw[u][0] &= keep[0];
                vw[u][1] &= keep[1];
                vw[u][2] &= keep[0];
                vw[u][3] &= keep[1];
            }
        }
        const bool mask = !there || t0 + KV_STEP - 1 > base || t0 < sp.len - a.window * (a.window > 0);
        f16x8_t pf[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float f = ks * cs[n];
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = s[n][e >> 2][e & 3] * f;
            if (mask) {
                const int t1 = t0 + 4 * g;  // the lane's first token
                if (a.tree) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int t = t1 + 16 * (e >> 2) + (e & 3);
                        const bool see = there & (t < sp.len) & ((t < base) | (((tree[n] >> ((t - base) & 31)) & 1u) != 0u));
                        x[e] = see ? x[e] : NEG_INF;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int t = t1 + 16 * (e >> 2) + (e & 3);
                        x[e] = there & (t <= pos[n]) & (t > lo[n]) ? x[e] : NEG_INF;
                    }
                }
            }
            float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
            if (__any(top > m[n] + 8.f)) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                // only the rows concerned: a row does not depend on its neighbours
                const float mn = top > m[n] + 8.f ? top : m[n];
                const float down = mn == NEG_INF ? 1.f : __builtin_amdgcn_exp2f(m[n] - mn);
                m[n] = mn;
                nm[n] = mn == NEG_INF ? 0.f : -mn;
                l[n] *= down;
                ps[n] *= down;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[n][d] *= down;
            }
            const float nr = nm[n] + lr;
#pragma unroll
            for (int e = 0; e < 8; ++e) pf[n][e] = (_Float16)__builtin_amdgcn_exp2f(x[e] + nr);
            // the sum of the step's p, as rounded, in every lane of the row
            const f32x4_t t = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pf[n], f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
            ps[n] += t[0];
            if (rr <= 8.f) {
                l[n] = fmaf(t[0], rr, l[n]);
            } else {
                // values far smaller than the chunk's largest: p vs / vref may
                // have left f16's range, so p is summed by itself
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += __builtin_amdgcn_exp2f(x[e] + nm[n]);
                sum += __shfl_xor(sum, 16);
                l[n] += sum + __shfl_xor(sum, 32);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const f16x8_t vf = codes8<E4M3>(vw[u][2 * d], vw[u][2 * d + 1]);
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    o[n][2 * u + d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[n], o[n][2 * u + d], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        load(vw, a.v, t0 + STRIDE);
    }
    // in true units
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const float back = -BIAS * ps[n];
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][d][e] = fmaf(o[n][d][e], UNIT, back) * vref;
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
                        for (int e = 0; e < 4; ++e) to[n * SL + 4 * d + e][lane] = o[n][d][e];
                    to[n * SL + DT * 4][lane] = m[n];
                    to[n * SL + DT * 4 + 1][lane] = l[n];
                }
            }
            __syncthreads();
            if (ts < half) {
                float(*from)[64] = slots[ts * RS + rsi];
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    const float m2 = from[n * SL + DT * 4][lane];
                    const float l2 = from[n * SL + DT * 4 + 1][lane];
                    const float mn = fmaxf(m[n], m2);
                    const float f1 = mn == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(m[n] - mn);
                    const float f2 = mn == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(m2 - mn);
                    m[n] = mn;
                    l[n] = l[n] * f1 + l2 * f2;
#pragma unroll
                    for (int d = 0; d < DT; ++d)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[n][d][e] = o[n][d][e] * f1 + from[n * SL + 4 * d + e][lane] * f2;
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
                    *reinterpret_cast<u32x2_t *>((uint16_t *)a.out + at + 16 * d) = bf16x4(v);
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

// Joins the chunks of one (query token, head).  D / 4 threads take 4
// dimensions each of one chunk; the workgroup's groups of them take the
// chunks in turn, four loads in flight a thread, and join in LDS.
constexpr int JOIN_T = 256;

template <int D>
__global__ void __launch_bounds__(JOIN_T) kv_attn_join_kernel(KvAttnArgs a) {
    constexpr int TD = D / 4, NG = JOIN_T / TD, AHEAD = 4;
    __shared__ f32x4_t so[NG][TD];
    __shared__ float sl[NG], smx[JOIN_T / 64];
    const int tid = threadIdx.x, gi = tid / TD, d4 = tid % TD;
    const int r = blockIdx.x / a.max_q, j = blockIdx.x % a.max_q, hq = blockIdx.y;
    const Span sp = span_of(a, r);
    if (j >= sp.T) return;
    const int row = a.q_start[r] + j;
    const int n = max(min(sp.c1 - sp.c0, a.chunks), 1);
    const size_t at = (size_t)row * a.Hq + hq, step = (size_t)a.M * a.Hq;
    float mx = NEG_INF;
    for (int c = tid; c < n; c += JOIN_T) mx = fmaxf(mx, a.part_ml[2 * (at + c * step)]);
#pragma unroll
    for (int d = 32; d; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
    if ((tid & 63) == 0) smx[tid >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < JOIN_T / 64; ++w) mx = fmaxf(mx, smx[w]);
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
    for (int c0 = gi; c0 < n; c0 += NG * AHEAD) {
        f32x4_t v[AHEAD];
        f32x2_t ml[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int c = min(c0 + i * NG, n - 1);
            v[i] = reinterpret_cast<const f32x4_t *>(a.part + (at + c * step) * D)[d4];
            ml[i] = reinterpret_cast<const f32x2_t *>(a.part_ml)[at + c * step];
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (c0 + i * NG >= n) break;
            // (a row of NaN scores has no maximum, but a NaN sum)
            const float f = mx == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(ml[i][0] - mx);
            l = fmaf(f, ml[i][1], l);
            o += v[i] * f;
        }
    }
    so[gi][d4] = o;
    if (d4 == 0) sl[gi] = l;
    __syncthreads();
    if (gi != 0) return;
#pragma unroll
    for (int k = 1; k < NG; ++k) {
        o += so[k][d4];
        l += sl[k];
    }
    const float f = sp.too_long ? __builtin_nanf("") : l == 0.f ? 0.f : 1.f / l;
    const size_t to = (size_t)row * a.out_stride + (size_t)hq * D + 4 * d4;
    o *= f;
    if (a.out_f32)
        *reinterpret_cast<f32x4_t *>((float *)a.out + to) = o;
    else
        *reinterpret_cast<u32x2_t *>((uint16_t *)a.out + to) = bf16x4(o);
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

template <bool E4M3, int D, int NR, int RS, int WAVES>
void run(const KvAttnArgs &a, hipStream_t s) {
    const int rows = a.max_q * a.G;
    const dim3 grid((unsigned)(a.R * a.Hkv * a.chunks), (unsigned)((rows + 16 * NR * RS - 1) / (16 * NR * RS)));
    hipLaunchKernelGGL((kv_attn_kernel<E4M3, D, NR, RS, WAVES>), grid, dim3(WAVES * 64), 0, s, a);
    if (a.chunks > 1)
        hipLaunchKernelGGL((kv_attn_join_kernel<D>), dim3((unsigned)(a.R * a.max_q), (unsigned)a.Hq), dim3(JOIN_T), 0, s, a);
}

template <bool E4M3, int D>
void pick(const KvAttnArgs &a, hipStream_t s) {
    const int rows = a.max_q * a.G;
    constexpr int NR = D == 256 ? 1 : 2;  // two row tiles of 256 dimensions do not fit the registers
    if (rows <= 16)
        run<E4M3, D, 1, 1, 4>(a, s);
    else if (rows <= 32)
        run<E4M3, D, NR, 2 / NR, 4>(a, s);
    else if (rows <= 64 || NR == 1)
        run<E4M3, D, NR, 4 / NR, 4>(a, s);
    else
        run<E4M3, D, NR, 4, 4>(a, s);
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
