// The attention kernel over the paged 8-bit cache (kv_attention.hip says how it
// works), as kv_attention.hip and kv_prefix.hip instantiate it.
#pragma once

#include <type_traits>

#include "kv_cache.h"

namespace qg {

// What a launch's line of work holds, and where its results go:
//   KV_PLAIN   the requests; the output, or segments where they are cut
//   KV_OWN     the requests; segments only, to be joined with the prefix's
//   KV_BOTH    the requests and, as one more entry, the prefix that they share:
//              all rows of the call against it, without masks; segments only
//   KV_PREFIX  the prefix alone, of kv_prefix_rows_kernel; segments only
//   KV_LAST    the requests, not cut, with the prefix's segments joined to them;
//              the output
enum KvMode { KV_PLAIN, KV_OWN, KV_BOTH, KV_PREFIX, KV_LAST };

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr float NEG_INF = -__builtin_inff();

// Probabilities are carried as 2^P_EXP p (in o, l and ps alike, so that it
// falls out of o / l): with p <= 2^8 that fills f16's range upwards, and what
// its normal range loses below starts at p vs / vref = 2^-21.
constexpr float P_EXP = 7.f, P_UNIT = 0x1p7f;

// A wave's o and l leave it in this unit (with P_UNIT's inverse in it): sums
// of p <= 2^8 over up to 2^16 tokens of values near fp32's end stay inside it,
// and the smallest scale that an append writes, 2^-109, keeps 16 bits.
constexpr float OUT_UNIT = 0x1p-31f;

// An int8 code c enters the MFMA as the f16 whose bits are c + 128: a
// denormal (which the MFMA keeps), worth (c + 128) 2^-24.  The products'
// accumulators are corrected by -128 times the other operand's sum, so their
// fp32 roundings are those of sums of up to 255: an output is off by up to
// about 2^-20 of 128 times its scale besides, also where all its codes are 0.
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

// What a request asks for: its T query tokens see the steps (of 32 tokens)
// from `start` on.
struct Req {
    int q0, T, len, start, units, groups;  // groups of RW rows
    bool too_long;                         // more tokens, or new ones, than the call was told of: its rows become NaN
    bool prefix;                           // the shared prefix: T are all rows of the call
    __device__ __forceinline__ int work(int Hkv) const { return units * groups * Hkv; }
};

// The kernel's arguments where the hardware left them, anew at each call: the
// compiler reads them again there instead of holding all of them in SGPRs,
// which are too few for that.
typedef const __attribute__((address_space(4))) KvAttnArgs Args;
__device__ __forceinline__ Args &args() {
    Args *p = (Args *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *p;
}

// entries of the line
template <KvMode MODE>
__device__ __forceinline__ int entries_of(Args &a) {
    return a.R + (MODE == KV_BOTH ? 1 : 0);
}

template <int RW, KvMode MODE = KV_PLAIN>
__device__ __forceinline__ Req req_of(Args &a, int r) {
    Req s;
    s.prefix = false;
    if (MODE == KV_PREFIX || (MODE == KV_BOTH && r == a.R)) {
        s.prefix = true;
        s.q0 = a.q_start[0];
        const int T = max((int)((unsigned)a.q_start[a.R] - (unsigned)s.q0), 0);
        s.T = s.q0 < 0 || s.q0 > a.M ? 0 : min(T, a.M - s.q0);
        const int held = max(a.prefix_len[0], 0);  // (of which the table may have fewer)
        s.len = min(held, a.prefix_blocks * a.page);
        s.too_long = held > a.max_prefix;
        s.start = 0;
        s.units = s.T == 0 ? 0 : s.too_long ? 1 : (s.len + KV_STEP - 1) / KV_STEP;
        s.groups = (s.T * a.G + RW - 1) / RW;
        return s;
    }
    s.q0 = a.q_start[r];
    const int T = max((int)((unsigned)a.q_start[r + 1] - (unsigned)s.q0), 0);
    s.T = min(T, a.max_q);
    if (s.q0 < 0 || s.q0 > a.M - s.T) s.T = 0;
    const int held = max(a.lens[r], 0);
    s.len = min(held, a.max_blocks * a.page);
    s.too_long = held > a.max_len || T > a.max_q;
    s.start = a.window > 0 ? max(s.len - s.T - a.window + 1, 0) & ~(KV_STEP - 1) : 0;
    s.units = s.T == 0 ? 0 : s.too_long ? 1 : max((s.len - s.start + KV_STEP - 1) / KV_STEP, 1);
    s.groups = (s.T * a.G + RW - 1) / RW;
    return s;
}

// Sum over the requests before `end` of their work, by the whole wave.
template <int RW, KvMode MODE = KV_PLAIN>
__device__ __forceinline__ int work_before(Args &a, int end, int lane) {
    if (end == 1) return __builtin_amdgcn_readfirstlane(req_of<RW, MODE>(a, 0).work(a.Hkv));
    int sum = 0;
    for (int r = lane; r < end; r += 64) sum += req_of<RW, MODE>(a, r).work(a.Hkv);
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    return __builtin_amdgcn_readfirstlane(sum);
}

// A workgroup's run, given all the work: equal runs, or, where a cut falls on
// every start (`aligned`), so long that the rounded-up parts fit too.
template <KvMode MODE = KV_PLAIN>
__device__ __forceinline__ int run_length(Args &a, int total) {
    const int starts = MODE == KV_PLAIN ? a.R * a.Hkv * a.groups : a.starts;
    const unsigned n = a.aligned ? a.slots - starts : a.slots;
    const int u = (int)(((unsigned)total + n - 1) / n);
    return (max(u, a.min_run) + a.min_run - 1) / a.min_run * a.min_run;
}

// The start of a line's segments in the workspace: the run's length and where each request's work
// starts on the line, for the second kernel.
constexpr int64_t PART_HEAD = 4 * (KV_R_MAX + 4);

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
                                                r, 16 * lane, (int)at + u * 1024, NT ? 2 : 0));
}

// Waves a SIMD that the registers are to leave room for.  Heads of 64 in E4M3 fit
// four, which the requests alone are to have (8 heads, 200 requests of up to 3000
// tokens 81 us against 87 of three, 48 of up to 16000 84 against 82); behind a prefix
// three are better (300 of up to 3000 behind 2000, 145 us against 154).
constexpr int attn_waves(bool e4m3, int D, int NR, int waves, KvMode mode) {
    return NR > 1 || D > 128 || waves != 4 ? 2 : e4m3 && D == 64 && mode == KV_PLAIN ? 4 : 3;
}

template <bool E4M3, int D, int NR, int RS, int WAVES, KvMode MODE = KV_PLAIN>
__global__ void __launch_bounds__(WAVES * 64, attn_waves(E4M3, D, NR, WAVES, MODE)) kv_attn_kernel(KvAttnArgs) {
    constexpr int TS = WAVES / RS;      // waves that split the tokens
    constexpr int KS = D / 32;          // MFMA steps of Q K^T
    constexpr int DT = D / 16;          // tiles of O
    constexpr int SL = DT * 4 + 2;      // floats a lane and row tile joins
    constexpr float UNIT = Code<E4M3>::unit, BIAS = Code<E4M3>::bias;
    constexpr int KB = D / 32;          // kilobytes of keys, and of values, of a step
    // Several waves that take different rows of the same tokens share a
    // step's codes through LDS; a wave alone reads them into its registers,
    // past the caches.
    constexpr bool SHARED = RS > 1;
    constexpr int PART = 2 * KB / RS;   // kilobytes each of them brings
    constexpr int STAGE = SHARED ? 2 * TS * 2 * KB * 64 : 0;
    constexpr int JOIN = TS > 1 ? (TS / 2) * RS * NR * SL * 16 : 0;
    __shared__ u32x4_t lds[STAGE > JOIN ? STAGE : JOIN > 0 ? JOIN : 1];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c = lane & 15;
    const int ts = wave / RS, rsi = wave % RS;
    constexpr int RW = 16 * NR * RS;
    const int shift = __builtin_ctz(args().page);
    const int per = args().Hkv * args().groups;  // (head, row group) pairs of a request

    // this workgroup's run [x, end) of the line, and the request it starts in
    int r, x, end, before;
    const bool whole = MODE == KV_LAST || (MODE == KV_PLAIN && args().whole);
    if (whole) {
        r = blockIdx.x / per;
        x = end = before = 0;
    } else {
        Args &a = args();
        int len = 0, unit = 1;  // steps are counted in `unit`s
        const int entries = entries_of<MODE>(a);
        len = run_length<MODE>(a, work_before<RW, MODE>(a, entries, lane));
        if (a.aligned) {
            unit = len;
            len = 1;
        }
        x = blockIdx.x * len;
        end = x + len;
        before = 0;
        r = -1;
        // the request that x falls into; the first workgroup goes through all
        // of them and leaves their starts for the second kernel
        const bool leave = blockIdx.x == 0 && wave == 0;
        if (leave && lane == 0) a.head[0] = a.aligned ? unit : len;
        int sum = 0;
        if (entries == 1) {
            const Req q = req_of<RW, MODE>(a, 0);
            if (x < (q.units + unit - 1) / unit * q.groups * a.Hkv) r = 0;
            if (leave && lane == 0) a.head[1] = 0;
        } else
            for (int r0 = 0; r0 < entries && (r < 0 || leave); r0 += 64) {
            int w = 0;
            if (r0 + lane < entries) {
                const Req q = req_of<RW, MODE>(a, r0 + lane);
                w = (q.units + unit - 1) / unit * q.groups * a.Hkv;
            }
            int upto = w;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int u = __shfl_up(upto, d);
                if (lane >= d) upto += u;
            }
            if (leave && r0 + lane < entries) a.head[1 + r0 + lane] = sum + upto - w;
            const unsigned long long past = __ballot(sum + upto > x);
            if (r < 0 && past) {
                const int i = __builtin_ctzll(past);
                r = r0 + i;
                before = sum + __builtin_amdgcn_readlane(upto - w, i);
            }
            sum += __builtin_amdgcn_readlane(upto, 63);
        }
        if (r < 0) return;
        if (a.aligned) end = -unit;  // one segment
    }
    for (;;) {  // segments
    Args &a = args();
    const Req rq = req_of<RW, MODE>(a, r);
    const int rows = rq.T * a.G;
    int h, rgi, u0, u1;
    if (whole) {
        const int pair = blockIdx.x % per;
        h = pair / a.groups;
        rgi = pair % a.groups;
        u0 = 0;
        u1 = rq.units;
        if (rgi * RW >= rows) return;
    } else {
        // (aligned: end = -(length of a segment), x counts segments)
        const int parts = end < 0 ? (rq.units - end - 1) / -end : rq.units;
        const int pair = (x - before) / parts, u = (x - before) % parts;
        h = pair / rq.groups;
        rgi = pair % rq.groups;
        u0 = end < 0 ? u * -end : u;
        u1 = min(rq.units, end < 0 ? u0 - end : u0 + end - x);
    }
    const bool all = u0 == 0 && u1 == rq.units;  // not cut
    const int row0 = rgi * RW, base = rq.len - (rq.prefix ? 1 : rq.T);  // base: position of the first query token
    const bool by_tree = a.tree != nullptr && !rq.prefix;
    const int t_begin = rq.start + u0 * KV_STEP, t_end = rq.too_long ? 0 : min(rq.start + u1 * KV_STEP, rq.len);

    // up to 64 pages from the step at t_lo on, and their scales, one a lane
    int t_lo = t_begin, t_hi = t_begin, page0 = 0, my_page = -1;
    float my_ks = 0.f, my_vs = 0.f, my_lr = 0.f, my_rr = 1.f, vref = 0.f;
    const auto pages = [&](int t) {
        t_lo = t;
        page0 = t >> shift;
        t_hi = min(t_end, (page0 + 64) << shift);
        my_page = -1;
        my_ks = my_vs = 0.f;
        if ((page0 + lane) << shift < t_hi) {
            my_page = rq.prefix ? a.prefix_table[page0 + lane] : a.table[(size_t)r * a.max_blocks + page0 + lane];
            if (my_page < 0 || my_page >= a.pages) my_page = -1;
            if (my_page >= 0) {
                my_ks = a.k_scales[(size_t)my_page * a.Hkv + h] * UNIT;
                my_vs = a.v_scales[(size_t)my_page * a.Hkv + h];
            }
        }
    };
    pages(t_begin);
    // N kilobytes of the step at t from `skip` on (past the end, or of a page
    // that is not there: none)
    const auto page_at = [&](int t) { return t < t_hi ? __builtin_amdgcn_readlane(my_page, (t >> shift) - page0) : -1; };
    const auto load = [&](auto &to, const uint8_t *codes, int t, unsigned skip) {
        const int page = page_at(t);
        const size_t at = ((size_t)max(page, 0) * a.Hkv + h) * ((size_t)a.page * D);
        load_codes<sizeof(to) / 16, !SHARED>(to, uniform_ptr(codes + at), page < 0 ? 0u : (unsigned)a.page * D,
                                             (unsigned)(t & (a.page - 1)) * D + skip, lane);
    };
    constexpr int STRIDE = TS * KV_STEP;
    u32x4_t kw[SHARED ? 1 : KB], vw[SHARED ? 1 : KB];    // a wave alone: one step
    u32x4_t st0[SHARED ? PART : 1], st1[SHARED ? PART : 1];  // sharing: its part of two steps
    const bool st_v = rsi * 2 >= RS;
    const uint8_t *st_codes = st_v ? a.v : a.k;
    const unsigned st_skip = 1024u * PART * (st_v ? rsi - RS / 2 : rsi);
    const auto first_loads = [&]() {
        const int first = t_lo + ts * KV_STEP;
        if constexpr (SHARED) {
            load(st0, st_codes, first, st_skip);
            load(st1, st_codes, first + STRIDE, st_skip);
        } else {
            load(kw, a.k, first, 0);
            load(vw, a.v, first, 0);
        }
    };
    first_loads();

    // Q, as f16 in the K tiles' order of dimensions
    f16x8_t qf[NR][KS];
    float cs[NR], k0[NR];  // factor and start of the scores
    int pos[NR], lo[NR];   // visible: lo < t <= pos
    unsigned tree[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int row = row0 + 16 * (rsi * NR + n) + c;
        const bool valid = row < rows;
        const int j = valid ? row / a.G : 0;
        const int hq = h * a.G + (valid ? row - j * a.G : 0);
        pos[n] = rq.prefix ? base : base + j;  // (every row sees all of a prefix)
        lo[n] = a.window > 0 ? pos[n] - a.window : -1;
        tree[n] = by_tree && valid ? a.tree[rq.q0 + j] : 0u;
        const uint16_t *q = a.q + (size_t)(rq.q0 + j) * a.q_stride + (size_t)hq * D;
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
        // (the codes' unit goes to the pages' scales: with it, large queries'
        // factor would leave fp32's range where the scores do not)
        cs[n] = ldexpf(fabsf(a.scale), -e2);
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

    // One step; MASK: some row may not see some of its tokens.  A wave alone
    // replaces its keys by the next step's once they are used, then its values: one buffer each, with loads in flight all the
    // time.  `buf`: where the shared codes lie.
    const auto compute = [&](auto masked, int t0, const u32x4_t *buf) {
        constexpr bool MASK = decltype(masked)::value;
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
                const int kb = i * (D / 64) + (k >> 1);
                const u32x4_t w = SHARED ? buf[kb * 64 + lane] : kw[SHARED ? 0 : kb];
                const f16x8_t kf = codes8<E4M3>(w[2 * (k & 1)], w[2 * (k & 1) + 1]);
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    s[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[n][k], s[n][i], 0, 0, 0);
            }
            if (k & 1) __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!SHARED) load(kw, a.k, t0 + STRIDE, 0);
        // codes of slots behind the last token may be anything (an E4M3 NaN),
        // and those of a page without a value scale are worth nothing
        unsigned keep[2] = {~0u, ~0u};
        if (no_v || (MASK && t0 + KV_STEP > rq.len)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                keep[i] = 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e) keep[i] |= ((t0 + 16 * i + 4 * g + e < rq.len) & !no_v) ? 0xFFu << (8 * e) : 0u;
            }
        }
        const float off = there ? 0.f : NEG_INF;
        f16x8_t pf[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float f = ks * cs[n];
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf(s[n][e >> 2][e & 3], f, off);
            if constexpr (MASK) {
                const int t1 = t0 + 4 * g;  // the lane's first token
                if (by_tree) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int t = t1 + 16 * (e >> 2) + (e & 3);
                        const bool see = (t < rq.len) & ((t < base) | (((tree[n] >> ((t - base) & 31)) & 1u) != 0u));
                        x[e] = see ? x[e] : NEG_INF;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int t = t1 + 16 * (e >> 2) + (e & 3);
                        x[e] = ((t <= pos[n]) & (t > lo[n])) ? x[e] : NEG_INF;
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
                l[n] = fmaf(sum + __shfl_xor(sum, 32), P_UNIT, l[n]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < KB; ++u) {
            u32x4_t w = SHARED ? buf[(KB + u) * 64 + lane] : vw[SHARED ? 0 : u];
            w[0] &= keep[0];
            w[1] &= keep[1];
            w[2] &= keep[0];
            w[3] &= keep[1];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const f16x8_t vf = codes8<E4M3>(w[2 * d], w[2 * d + 1]);
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    o[n][2 * u + d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[n], o[n][2 * u + d], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!SHARED) load(vw, a.v, t0 + STRIDE, 0);
    };
    if constexpr (TS > 1 || SHARED) __syncthreads();  // LDS is free of the last segment
    while (t_lo < t_end) {  // windows of 64 pages
        // every row sees all of the steps before this one (the first new token
        // only where there is no tree)
        const int t_clear = a.window > 0 ? t_lo : min(t_hi, (base + (by_tree ? 0 : 1)) & ~(KV_STEP - 1));
        // vref: a power of two at least as large as every value scale so far (0
        // before the first: a page whose values are all 0 has none, and what it
        // left in o and ps is nothing but the codes' bias, which f = 0 clears);
        // a page's scale over it, as a power of two in the exponent, and its
        // inverse
        float up = fmaxf(my_vs, 0.f);
#pragma unroll
        for (int d = 32; d; d >>= 1) up = fmaxf(up, __shfl_xor(up, d));
        up = readlane_f(up, 0);
        if (up > vref) {
            up = pow2_above(up);
            const float f = vref / up;
            vref = up;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                ps[n] *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[n][d] *= f;
            }
        }
        my_lr = (my_vs > 0.f ? __builtin_amdgcn_logf(my_vs / vref) : 0.f) + P_EXP;
        my_rr = my_vs > 0.f ? vref / my_vs : 1.f;
        if constexpr (SHARED) {
            // two steps' parts in registers, two in LDS: a part is written to
            // LDS while the next one's loads run, and one barrier a step tells
            // that all parts are there (and that the step before the last is
            // used up)
            u32x4_t *mine = lds + (ts * 2 * KB + (st_v ? KB : 0)) * 64 + (st_skip / 16) + lane;
            const auto stage = [&](auto masked, u32x4_t(&st)[PART], int t, int b) {
                u32x4_t *to = mine + b * (TS * 2 * KB * 64);
#pragma unroll
                for (int u = 0; u < PART; ++u) to[u * 64] = st[u];
                load(st, st_codes, t + 2 * STRIDE, st_skip);
                __syncthreads();
                if (t < t_hi) compute(masked, t, lds + (b * TS + ts) * 2 * KB * 64);
            };
            int t0 = t_lo;
            for (; t0 + 2 * STRIDE <= t_clear; t0 += 2 * STRIDE) {
                stage(std::false_type(), st0, t0 + ts * KV_STEP, 0);
                stage(std::false_type(), st1, t0 + STRIDE + ts * KV_STEP, 1);
            }
            for (; t0 < t_hi; t0 += 2 * STRIDE) {
                stage(std::true_type(), st0, t0 + ts * KV_STEP, 0);
                stage(std::true_type(), st1, t0 + STRIDE + ts * KV_STEP, 1);
            }
        } else {
            int t0 = t_lo + ts * KV_STEP;
            for (; t0 < t_clear; t0 += STRIDE) compute(std::false_type(), t0, nullptr);
            for (; t0 < t_hi; t0 += STRIDE) compute(std::true_type(), t0, nullptr);
        }
        if (t_hi >= t_end) break;
        pages(t_hi);
        first_loads();
    }
    // o in OUT_UNITs
    const float out_unit = vref * OUT_UNIT;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const float back = -BIAS * ps[n];
        l[n] = MODE != KV_PLAIN && rq.too_long ? __builtin_nanf("") : l[n] * OUT_UNIT;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][d][e] = fmaf(o[n][d][e], UNIT, back) * out_unit;
    }
    // the prefix's segments, spread over the waves that split the tokens
    if constexpr (MODE == KV_LAST) {
        Args &a = args();
        const Req pq = req_of<RW, KV_PREFIX>(a, 0);
        const int cut = max(a.pre_head[0], 1), segs = pq.units > 0 ? (pq.units + cut - 1) / cut : 0;
        const int pgroups = (pq.T * a.G + a.pre_rw - 1) / a.pre_rw;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int row = (rq.q0 - pq.q0) * a.G + min(row0 + 16 * (rsi * NR + n) + c, rows - 1);
            const int slot = (h * pgroups + row / a.pre_rw) * segs;
            // (so of q_start out of order only, or if another call wrote to the workspace)
            if (row < 0 || row >= pq.T * a.G || segs > a.pre_slots || slot > a.pre_slots - segs) continue;
            const size_t at = (size_t)slot * a.pre_rows + row % a.pre_rw;
            for (int i = ts; i < segs; i += TS) {
                const size_t from = at + (size_t)i * a.pre_rows;
                const f32x2_t ml = *reinterpret_cast<const f32x2_t *>(a.pre_ml + 2 * from);
                f32x4_t v[DT];
#pragma unroll
                for (int d = 0; d < DT; ++d) v[d] = *reinterpret_cast<const f32x4_t *>(a.pre_part + from * D + 16 * d + 4 * g);
                const float mn = fmaxf(m[n], ml[0]);
                const float f1 = mn == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(m[n] - mn);
                const float f2 = mn == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(ml[0] - mn);
                m[n] = mn;
                l[n] = l[n] * f1 + ml[1] * f2;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[n][d] = o[n][d] * f1 + v[d] * f2;
            }
        }
    }
    // join the waves that split the tokens, half of them at a time
    if constexpr (TS > 1) {
#pragma unroll
        for (int half = TS / 2; half; half >>= 1) {
            __syncthreads();
            if (ts >= half && ts < 2 * half) {
                float(*to)[64] = reinterpret_cast<float(*)[64]>(lds) + ((ts - half) * RS + rsi) * (NR * SL);
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
                float(*from)[64] = reinterpret_cast<float(*)[64]>(lds) + (ts * RS + rsi) * (NR * SL);
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
    if (ts == 0) {
        Args &a = args();
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int row = row0 + 16 * (rsi * NR + n) + c;
            if (row >= rows) continue;
            if (MODE == KV_LAST || (MODE == KV_PLAIN && all)) {
                const float f = rq.too_long ? __builtin_nanf("") : l[n] == 0.f ? 0.f : 1.f / l[n];
                const int j = row / a.G;
                const size_t at = (size_t)(rq.q0 + j) * a.out_stride + (size_t)(h * a.G + row - j * a.G) * D + 4 * g;
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const f32x4_t v = o[n][d] * f;
                    if (a.out_f32)
                        *reinterpret_cast<f32x4_t *>((float *)a.out + at + 16 * d) = v;
                    else
                        *reinterpret_cast<u32x2_t *>((uint16_t *)a.out + at + 16 * d) = bf16x4(v);
                }
            } else {
                // its place: segments and pairs both only go up along the line
                const size_t at = (size_t)(blockIdx.x + (end < 0 ? 0 : r * per + h * rq.groups + rgi)) * a.part_rows + 16 * (rsi * NR + n) + c;
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    *reinterpret_cast<f32x4_t *>(a.part + at * D + 16 * d + 4 * g) = o[n][d];
                if (g == 0) *reinterpret_cast<f32x2_t *>(a.part_ml + 2 * at) = f32x2_t{m[n], l[n]};
            }
        }
    }
    if (whole) return;
    x += u1 - u0;
    if (x >= end) return;  // (aligned: end < 0)
    if (x - before >= rq.work(a.Hkv)) {  // on to the next request that has work
        before = x;
        do ++r;
        while (r < entries_of<MODE>(a) && req_of<RW, MODE>(a, r).units == 0);
        if (r >= entries_of<MODE>(a)) return;
    }
    }
}

namespace {

// Where one row's part of a segment lies: its place among a line's part and part_ml.
struct Part {
    const float *part, *ml;
    size_t at;
};

template <int D, int W>
struct JoinLds {
    f32x4_t o[W > 1 ? W : 1][D / 4];
    float l[W], m[W];
};

// The output of (row, hq) from its n segments, part_at(c) the c-th, by W waves
// (wi: this one).  D / 4 lanes take 4 dimensions each of one segment; the
// waves' groups of them take the segments in turn, eight loads in flight a
// lane, and join across lanes and in LDS.  The maximum runs along with the
// sums (read in a pass before them: 128 rows 10.8 us against 10.2, 64 rows 7.8
// against 7.4).
template <int D, int W, typename At>
__device__ __forceinline__ void join_segments(Args &a, JoinLds<D, W> &lds, int n, int row, int hq, int wi, int lane, At part_at) {
    constexpr int TD = D / 4, NG = W * 64 / TD, AHEAD = 8;
    const int tid = wi * 64 + lane, gi = tid / TD, d4 = tid % TD;
    // with a running maximum, so that values and maxima are loaded together
    float mx = NEG_INF;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
    for (int c0 = gi; c0 < n; c0 += NG * AHEAD) {
        f32x4_t v[AHEAD];
        f32x2_t ml[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int c = min(c0 + i * NG, n - 1);
            const Part p = part_at(c);
            v[i] = *reinterpret_cast<const f32x4_t *>(p.part + p.at * D + 4 * d4);
            ml[i] = *reinterpret_cast<const f32x2_t *>(p.ml + 2 * p.at);
        }
        float mn = mx;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) mn = fmaxf(mn, ml[i][0]);
        const float down = mn == NEG_INF ? 1.f : __builtin_amdgcn_exp2f(mx - mn);
        mx = mn;
        l *= down;
        o *= down;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            // (a row of NaN scores has no maximum, but a NaN sum)
            const float f = mx == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(ml[i][0] - mx);
            if (c0 + i * NG < n) {
                l = fmaf(f, ml[i][1], l);
                o += v[i] * f;
            }
        }
    }
    // the wave's groups of lanes, then the waves
    float top = mx;
#pragma unroll
    for (int d = TD; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float down = top == NEG_INF ? 1.f : __builtin_amdgcn_exp2f(mx - top);
    l *= down;
    o *= down;
#pragma unroll
    for (int d = TD; d < 64; d <<= 1) {
        l += __shfl_xor(l, d);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], d);
    }
    if constexpr (W > 1) {
        if (lane < TD) lds.o[wi][lane] = o;
        if (lane == 0) {
            lds.l[wi] = l;
            lds.m[wi] = top;
        }
        __syncthreads();
        if (wi != 0) return;
        const float mine = top;
#pragma unroll
        for (int k = 1; k < W; ++k) top = fmaxf(top, lds.m[k]);
        const float own = top == NEG_INF ? 1.f : __builtin_amdgcn_exp2f(mine - top);
        o *= own;
        l *= own;
#pragma unroll
        for (int k = 1; k < W; ++k) {
            const float f = top == NEG_INF ? 1.f : __builtin_amdgcn_exp2f(lds.m[k] - top);
            o += lds.o[k][lane % TD] * f;
            l = fmaf(lds.l[k], f, l);
        }
    }
    if (lane >= TD) return;
    const float f = l == 0.f ? 0.f : 1.f / l;
    const size_t to = (size_t)row * a.out_stride + (size_t)hq * D + 4 * d4;
    o *= f;
    if (a.out_f32)
        *reinterpret_cast<f32x4_t *>((float *)a.out + to) = o;
    else
        *reinterpret_cast<u32x2_t *>((uint16_t *)a.out + to) = bf16x4(o);
}

// The variant for a call's rows (query tokens * heads to a KV head): row tiles
// a wave holds, waves that take different rows.
struct Shape {
    int NR, RS;
};

constexpr Shape shape_of(int D, int64_t rows) {
    if (rows <= 16) return {1, 1};
    if (D == 256) return {1, rows <= 32 ? 2 : 4};  // two row tiles of 256 dimensions do not fit the registers
    return {2, rows <= 32 ? 1 : rows <= 64 ? 2 : 4};
}

}  // namespace

}  // namespace qg
