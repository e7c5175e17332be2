// Attention of requests that share a prefix: as kv_attention.hip, with the
// prefix's tokens read once for all rows of the call.
//
// A row's softmax runs over the prefix and over its request's own tokens; both
// leave (maximum, sum, values) segments, and a join makes them one.  Against
// the prefix all query tokens of all requests are rows of one product, so what
// is memory's work for one request becomes the matrix cores' for many.  Up to
// 16 rows to a KV head the prefix is one more entry on the requests' line of
// work, in one launch; above it is a line of its own, of groups of up to 128
// rows times equal parts of the prefix.  What joins the segments is a kernel, or
// the requests' own one (KV_LAST), whichever costs less (kv_prefix_plan).
//
// Measured (eager calls one after another, 8 KV heads of 128 unless said; the rules'
// figures below are whole calls in a captured graph): 4 requests of 4 rows behind 8192
// tokens 18.5 us (12.8 the line, 6.2 the join: latency, a chain of loads before the
// first step and after the last; 17.4 in a graph); 48 behind 32768 73 us (47.5 the prefix, 510 TFLOP/s;
// 28 the requests, up to 2000 own tokens); 256 drafts of 16 requests, 1024 rows a
// head, behind 20011 110 us (94 the prefix, 715 TFLOP/s; 29 the requests, of which 6
// join, latency); 8 requests, 4 heads of 256, E4M3, behind 131072 87 us (61 the
// prefix, 4.4 TB/s and 560 TFLOP/s; 11.7 the requests, 13 the join, of 33 MB of
// segments); 32 requests behind 333 tokens 18.0 us.  Read for each request by
// kv_attention_run, 48 times 32768 tokens are 3.2 GB.
#include "kv_attn_kernel.h"

namespace qg {

struct KvPrefixJoinArgs {
    KvAttnArgs own, pre;
    int own_rw, pre_rw;  // rows of a group
    bool both;
};

namespace {

// Where an entry's segments lie for one of its rows.
struct Segments {
    int n;
    size_t at, step;  // rows of the parts
};

__device__ __forceinline__ Segments segments_of(const KvAttnArgs &a, const Req &rq, int entry, int before, int len, int rw,
                                                int head, int row, bool aligned, int per) {
    Segments s{0, 0, (size_t)a.part_rows};
    // (rows out of the entry's: of q_start out of order only)
    if (rq.units <= 0 || row < 0 || row >= rq.T * a.G) return s;
    const int groups = (rq.T * a.G + rw - 1) / rw, pair = head * groups + row / rw;
    int slot;
    if (aligned) {
        s.n = (rq.units + len - 1) / len;
        slot = before + pair * s.n;
    } else {
        const int x = before + pair * rq.units;
        slot = x / len;
        s.n = (x + rq.units - 1) / len - slot + 1;
        slot += entry * per + pair;
    }
    // (never so, unless another call wrote to the workspace in between)
    if (slot < 0 || s.n < 1 || s.n > a.part_slots || slot > a.part_slots - s.n) s.n = 0;
    s.at = (size_t)slot * a.part_rows + row % rw;
    return s;
}

// Joins the segments of a (query token, head), its request's and the prefix's: W waves for each.
template <int D, int W>
__global__ void __launch_bounds__(512) kv_prefix_join_kernel(KvPrefixJoinArgs p) {
    constexpr int ROWS = 8 / W;
    __shared__ JoinLds<D, W> lds;
    Args &a = *(Args *)__builtin_amdgcn_kernarg_segment_ptr();
    Args &b = *((Args *)__builtin_amdgcn_kernarg_segment_ptr() + 1);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = wave % W;
    const int which = blockIdx.x * ROWS + wave / W;  // (request, token, head)
    const int r = which / (a.max_q * a.Hq), j = which / a.Hq % a.max_q, hq = which % a.Hq;
    if (r >= a.R) return;
    const Req rq = req_of<16, KV_OWN>(a, r), pq = req_of<16, KV_PREFIX>(b, 0);
    if (j >= rq.T) return;
    const int head = hq / a.G, g = hq % a.G, prow = (rq.q0 - pq.q0 + j) * a.G + g;
    const Segments s = segments_of(p.own, rq, r, a.head[1 + r], max(a.head[0], 1), p.own_rw, head, j * a.G + g, a.aligned, a.Hkv * a.groups);
    Segments t = p.both ? segments_of(p.own, pq, a.R, a.head[1 + a.R], max(a.head[0], 1), p.own_rw, head, prow, a.aligned, a.Hkv * a.groups)
                        : segments_of(p.pre, pq, 0, 0, pq.units > 0 ? max(b.head[0], 1) : 1, p.pre_rw, head, prow, true, 0);
    const float *part = p.both ? a.part : b.part, *part_ml = p.both ? a.part_ml : b.part_ml;
    const int n = s.n + t.n;
    join_segments<D, W>(a, lds, n, rq.q0 + j, hq, wi, lane, [&](int c) {
        const bool own = c < s.n;
        return Part{own ? a.part : part, own ? a.part_ml : part_ml, own ? s.at + c * s.step : t.at + (c - s.n) * t.step};
    });
}

// The prefix against many rows: a workgroup of WAVES waves takes 16 NR WAVES
// rows of a KV head and one of the prefix's parts.  The waves convert a step's
// codes (32 tokens) to f16 once for all of them, into LDS, keys one step ahead
// of values: a step's scores are made by the matrix cores while the softmax of
// the step before is on the vector unit.  Nothing is masked but what lies
// behind the prefix's last token.
//
// A score times its factor less the row's maximum is one FMA, whose product is exact
// where the maximum's was rounded: by up to 2^-24 of the score the largest token's power
// is not 1, which for scores past LARGEST would leave f16 (from about 2^27 on rows were 0
// or NaN).  Rows that may have such scores round the product first, as the requests'
// kernel does, in masked steps; which rows those are goes by their own queries and the
// window's key scales, so no other row's bits depend on it.
//
// Four waves of 32 rows, two workgroups a CU (1024 rows a head 95.4 us, one of eight
// waves 99.6: all of them wait at every step's barrier); 16 rows a wave where rows are
// few (prefix_shape); 64 rows a wave leave one wave a SIMD (196 us).  What an unmasked
// step does besides its products was most of its time: staging with branches 105 us,
// without 95; before the first product 97, under the second 93.  A step of the two
// waves of a SIMD then takes about 2050 clocks, of which the matrix unit is busy for
// half, and the clock is near 1.5 GHz under such work (a library product of 8192 cubed
// reaches 1.4 of the 2.5 PFLOP/s); keys read a step earlier changed nothing.
template <bool E4M3, int D, int NR, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, 2) kv_prefix_rows_kernel(KvAttnArgs) {
    constexpr int KS = D / 32, DT = D / 16, KB = D / 32;
    constexpr int PW = 2 * KB / WAVES;  // kilobytes of codes that a wave brings of a step
    static_assert(PW >= 1 && PW * WAVES == 2 * KB, "half of the waves bring keys, half values");
    constexpr float UNIT = Code<E4M3>::unit, BIAS = Code<E4M3>::bias;
    // a score is at most this times its factor: D codes times queries of up to 2^14
    constexpr float REACH = D * 0x1p14f * (E4M3 ? 448.f : 128.f) / UNIT, LARGEST = 0x1p22f;
    __shared__ u32x4_t kbuf[2][2 * KB * 64], vbuf[2][2 * KB * 64];
    __shared__ float reach[WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c = lane & 15;
    constexpr int RW = 16 * NR * WAVES;
    Args &a = args();
    const Req rq = req_of<RW, KV_PREFIX>(a, 0);
    const int rows = rq.T * a.G;
    // heads fastest: the workgroups of a head, which read the same codes, run
    // on one XCD where there are eight heads
    const int h = blockIdx.x % a.Hkv, cut = blockIdx.x / a.Hkv % a.cuts, rg = blockIdx.x / a.Hkv / a.cuts;
    const int len = (rq.units + a.cuts - 1) / a.cuts;
    if (blockIdx.x == 0 && tid == 0) {
        a.head[0] = len;
        a.head[1] = 0;
    }
    if (rg >= rq.groups || cut * len >= rq.units) return;
    const int shift = __builtin_ctz(a.page);
    const int t_begin = cut * len * KV_STEP, t_end = rq.too_long ? 0 : min((cut + 1) * len * KV_STEP, rq.len);
    const int row0 = rg * RW + 16 * NR * wave;

    // Q, as f16 in the K tiles' order of dimensions
    f16x8_t qf[NR][KS];
    float cs[NR], k0[NR];  // factor and start of the scores
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int row = row0 + 16 * n + c;
        const bool valid = row < rows;
        const int j = valid ? row / a.G : 0;
        const int hq = h * a.G + (valid ? row - j * a.G : 0);
        const uint16_t *q = a.q + (size_t)(rq.q0 + j) * a.q_stride + (size_t)hq * D;
        u32x4_t w[KS];
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            w[s] = *reinterpret_cast<const u32x4_t *>(q + 64 * (s >> 1) + 16 * g + 8 * (s & 1));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const unsigned u = w[s][e];
                top = fmaxf(top, fmaxf(fabsf(bf16_lo(u)), fabsf(bf16_hi(u))));
            }
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
                const unsigned u = w[s][e >> 1];
                const float x = ldexpf(e & 1 ? bf16_hi(u) : bf16_lo(u), e2);
                const _Float16 hx = (_Float16)(a.scale < 0.f ? -x : x);
                qf[n][s][e] = hx;
                sum += (float)hx;
            }
        if (BIAS != 0.f) {
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
        }
        k0[n] = -(BIAS / UNIT) * sum;
        cs[n] = top > 0.f ? ldexpf(fabsf(a.scale), -e2) : 0.f;
    }
    // the wave's largest factor
    float most_cs = cs[0];
#pragma unroll
    for (int n = 1; n < NR; ++n) most_cs = fmaxf(most_cs, cs[n]);
#pragma unroll
    for (int d = 8; d; d >>= 1) most_cs = fmaxf(most_cs, __shfl_xor(most_cs, d));
    if (lane == 0) reach[wave] = most_cs;

    f32x4_t o[NR][DT], s[NR][2];
    float m[NR], nm[NR], l[NR], ps[NR], vref = 0.f;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        m[n] = NEG_INF;
        nm[n] = l[n] = ps[n] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    const f16x8_t ones = {(_Float16)1.f, (_Float16)1.f, (_Float16)1.f, (_Float16)1.f,
                          (_Float16)1.f, (_Float16)1.f, (_Float16)1.f, (_Float16)1.f};
    const bool brings_v = wave >= WAVES / 2;
    const unsigned skip = 1024u * PW * (wave % (WAVES / 2));
    const uint8_t *codes = brings_v ? a.v : a.k;

    for (int w0 = t_begin; w0 < t_end;) {  // windows of 64 pages, one a lane
        const int page0 = w0 >> shift;
        const int w1 = (int)min((int64_t)t_end, (int64_t)(page0 + 64) << shift);
        const int steps = (w1 - w0 + KV_STEP - 1) / KV_STEP;
        int my_page = -1;
        float my_ks = 0.f, my_vs = 0.f;
        if (page0 + lane <= (w1 - 1) >> shift) {
            my_page = a.prefix_table[page0 + lane];
            if (my_page < 0 || my_page >= a.pages) my_page = -1;
            if (my_page >= 0) {
                my_ks = a.k_scales[(size_t)my_page * a.Hkv + h] * UNIT;
                my_vs = a.v_scales[(size_t)my_page * a.Hkv + h];
            }
        }
        // vref: a power of two at least as large as every value scale so far
        float up = fmaxf(my_vs, 0.f), most_ks = my_ks;
#pragma unroll
        for (int d = 32; d; d >>= 1) {
            up = fmaxf(up, __shfl_xor(up, d));
            most_ks = fmaxf(most_ks, __shfl_xor(most_ks, d));
        }
        up = readlane_f(up, 0);
        most_ks = readlane_f(most_ks, 0) * REACH;
        if (up > vref) {
            up = pow2_above(up);
            const float down = vref / up;
            vref = up;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                ps[n] *= down;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[n][d] *= down;
            }
        }
        // of a page: log2 of the value scale's part of vref (-infinity where there
        // is no page), and its inverse (0: no value scale)
        const float my_lr = my_page < 0 ? NEG_INF : (my_vs > 0.f ? __builtin_amdgcn_logf(my_vs / vref) : 0.f) + P_EXP;
        const float my_rr = my_vs > 0.f ? vref / my_vs : 0.f;
        // where a wave's part of the page lies, and how much of it there is
        const uint64_t my_at = reinterpret_cast<uint64_t>(codes) + ((size_t)max(my_page, 0) * a.Hkv + h) * ((size_t)a.page * D) + skip;
        const unsigned my_lo = (unsigned)my_at, my_hi = (unsigned)(my_at >> 32), my_bytes = my_page < 0 ? 0u : (unsigned)a.page * D - skip;
        // whether every page is there, has a value scale, and one whose part of
        // vref leaves p in f16's range
        const bool plain = !__any(page0 + lane <= (w1 - 1) >> shift && !(my_rr > 0.f && my_rr <= 8.f));
        const auto page_of = [&](int i) { return ((w0 + min(i, steps - 1) * KV_STEP) >> shift) - page0; };
        __syncthreads();  // LDS is free of the last window (and every wave's reach is there)
        // this wave's part of step i (of the last one again where i is past it)
        const auto load = [&](u32x4_t(&to)[PW], int i) {
            const int page = page_of(i), t = w0 + min(i, steps - 1) * KV_STEP;
            const uint64_t at = (uint64_t)(unsigned)__builtin_amdgcn_readlane((int)my_lo, page) |
                                ((uint64_t)(unsigned)__builtin_amdgcn_readlane((int)my_hi, page) << 32);
            load_codes<PW, false>(to, reinterpret_cast<const uint8_t *>(at), (unsigned)__builtin_amdgcn_readlane((int)my_bytes, page),
                                  (unsigned)(t & (a.page - 1)) * D, lane);
        };
        // its codes, converted, to LDS
        u32x4_t *const home = (brings_v ? vbuf[0] : kbuf[0]) + skip / 8 + lane;  // (1024 bytes of codes: 128 operands)
        const auto store = [&](auto masked, u32x4_t(&st)[PW], int i) {
            if (decltype(masked)::value && brings_v) {
                // codes of slots behind the last token may be anything (an E4M3
                // NaN), those of a page without a value scale are worth nothing
                const int t = w0 + i * KV_STEP + 4 * g;
                const bool no_v = readlane_f(my_rr, page_of(i)) == 0.f;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    unsigned keep = 0u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) keep |= ((t + 16 * half + e < rq.len) & !no_v) ? 0xFFu << (8 * e) : 0u;
#pragma unroll
                    for (int u = 0; u < PW; ++u) {
                        st[u][half] &= keep;
                        st[u][2 + half] &= keep;
                    }
                }
            }
            u32x4_t *to = home + (i & 1) * (2 * KB * 64);
#pragma unroll
            for (int u = 0; u < PW; ++u) {
                to[2 * u * 64] = __builtin_bit_cast(u32x4_t, codes8<E4M3>(st[u][0], st[u][1]));
                to[(2 * u + 1) * 64] = __builtin_bit_cast(u32x4_t, codes8<E4M3>(st[u][2], st[u][3]));
            }
        };
        // operand q of the step's keys, and of its values
        const auto key = [&](const u32x4_t *buf, int q) { return __builtin_bit_cast(f16x8_t, buf[q * 64 + lane]); };
        const auto start = [&](int n) { return f32x4_t{k0[n], k0[n], k0[n], k0[n]}; };
        // of step i, whose scores are in s: the factor to them, and a
        // lane's largest of each row
        float f[NR], top[NR];
        const auto sees = [&](int i, int e) { return w0 + i * KV_STEP + 4 * g + 16 * (e >> 2) + (e & 3) < rq.len; };
        bool large = false;  // whether any of the workgroup's rows may have large scores
        const auto largest = [&](auto masked, int i) {
            const float ks = readlane_f(my_ks, page_of(i));
            const bool there = !decltype(masked)::value || __builtin_amdgcn_readlane(my_page, page_of(i)) >= 0;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                f[n] = ks * cs[n];
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = !decltype(masked)::value || sees(i, e) ? s[n][e >> 2][e & 3] : NEG_INF;
                const float most = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
                top[n] = !decltype(masked)::value || (there && most > NEG_INF) ? most * f[n] : NEG_INF;
                if (decltype(masked)::value && large && !(cs[n] * most_ks <= LARGEST)) {
                    s[n][0] *= f[n];
                    s[n][1] *= f[n];
                    f[n] = 1.f;
                }
            }
        };
        // step i: keys of i + 1 and values of i are in LDS, scores of i in s.
        // What the wave brings next (keys of i + 2, values of i + 1) goes there
        // meanwhile, and what comes two steps later is asked for.  Matrix
        // instructions take four times a vector instruction's time, so they are
        // spread: the next scores among the powers, the sums among the next
        // scores' maxima and the conversions.  `masked`: step i + 1 may end behind the last token.
        const auto step = [&](auto masked, u32x4_t(&st)[PW], int i) {
            const float lr = readlane_f(my_lr, page_of(i)), rr = readlane_f(my_rr, page_of(i));
            __syncthreads();
            constexpr int NK = 2 * KS, HELD = NK < 8 ? NK : 8;  // operands of keys; as many are read ahead
            const u32x4_t *kb = kbuf[(i + 1) & 1], *vb = vbuf[i & 1];
            f16x8_t kf[HELD], vf[HELD];
#pragma unroll
            for (int q = 0; q < HELD; ++q) kf[q] = key(kb, q);
            __builtin_amdgcn_sched_barrier(0);
            bool rise = false;
#pragma unroll
            for (int n = 0; n < NR; ++n) rise |= top[n] > m[n] + 8.f;
            if (__any(rise)) {
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    top[n] = fmaxf(top[n], __shfl_xor(top[n], 16));
                    top[n] = fmaxf(top[n], __shfl_xor(top[n], 32));
                    // only the rows concerned: a row does not depend on its neighbours
                    const float mn = top[n] > m[n] + 8.f ? top[n] : m[n];
                    const float down = mn == NEG_INF ? 1.f : __builtin_amdgcn_exp2f(m[n] - mn);
                    m[n] = mn;
                    nm[n] = mn == NEG_INF ? 0.f : -mn;
                    l[n] *= down;
                    ps[n] *= down;
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[n][d] *= down;
                }
            }
            if (decltype(masked)::value && !(rr > 0.f && rr <= 8.f) && lr > NEG_INF) {
                // values far smaller than the largest: p vs / vref may have left
                // f16's range, so p is summed by itself
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    float sum = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sum += !decltype(masked)::value || sees(i, e) ? __builtin_amdgcn_exp2f(fmaf(s[n][e >> 2][e & 3], f[n], nm[n])) : 0.f;
                    sum += __shfl_xor(sum, 16);
                    l[n] = fmaf(sum + __shfl_xor(sum, 32), P_UNIT, l[n]);
                }
            }
            f32x4_t was[NR][2];  // scores of step i
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                was[n][0] = s[n][0];
                was[n][1] = s[n][1];
            }
            const int ahead = brings_v ? i + 1 : i + 2;
            if (decltype(masked)::value) store(masked, st, ahead);
            __builtin_amdgcn_sched_barrier(0);
            // operand q: token tile (q / 2) / (D / 64), MFMA step the rest
#pragma unroll
            for (int q = 0; q < NK; ++q) {
                const int t = q / KS, k = q % KS;
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    s[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[q % HELD], qf[n][k], k == 0 ? start(n) : s[n][t], 0, 0, 0);
                if (q + HELD < NK) kf[q % HELD] = key(kb, q + HELD);
                if (q >= NK - HELD) vf[q - (NK - HELD)] = key(vb, q - (NK - HELD));
            }
            f16x8_t pf[NR];
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const float nr = nm[n] + lr;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = fmaf(was[n][e >> 2][e & 3], f[n], nr);
                    pf[n][e] = (_Float16)__builtin_amdgcn_exp2f(!decltype(masked)::value || sees(i, e) ? x : NEG_INF);
                }
            }
#pragma unroll
            for (int r = 0; r < NK; ++r) {
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
                    __builtin_amdgcn_sched_group_barrier(0x400, 8 / NK, 0);
                }
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (!decltype(masked)::value) store(masked, st, ahead);
            load(st, ahead + 2);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
#pragma unroll
                for (int n = 0; n < NR; ++n) o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[d % HELD], pf[n], o[n][d], 0, 0, 0);
                if (d + HELD < DT) vf[d % HELD] = key(vb, d + HELD);
            }
            f32x4_t t[NR];  // the sum of the step's p, as rounded, in every lane of the row
#pragma unroll
            for (int n = 0; n < NR; ++n) t[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pf[n], f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
            largest(masked, i + 1);
#pragma unroll
            for (int r = 0; r < DT; ++r) {
                __builtin_amdgcn_sched_group_barrier(0x008, NR, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 2 * NR, 0);
            }
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                ps[n] += t[n][0];
                if (!decltype(masked)::value || (rr > 0.f && rr <= 8.f)) l[n] = fmaf(t[n][0], rr, l[n]);
            }
        };
        u32x4_t st0[PW], st1[PW];
        load(st0, 0);
        load(st1, 1);
#pragma unroll
        for (int w = 0; w < WAVES; ++w) large |= !(readlane_f(reach[w], 0) * most_ks <= LARGEST);
        store(std::true_type(), st0, 0);
        if (!brings_v) store(std::true_type(), st1, 1);
        load(st0, brings_v ? 1 : 2);
        load(st1, brings_v ? 2 : 3);
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 2 * KS; ++q)
#pragma unroll
            for (int n = 0; n < NR; ++n)
                s[n][q / KS] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key(kbuf[0], q), qf[n][q % KS], q % KS == 0 ? start(n) : s[n][q / KS], 0, 0, 0);
        largest(std::true_type(), 0);
        const int clear = plain && !large ? (w1 - w0) / KV_STEP - 1 : 0;  // steps before a whole one
        int i = 0;
        for (; i + 2 <= clear; i += 2) {
            step(std::false_type(), st0, i);
            step(std::false_type(), st1, i + 1);
        }
        for (; i < steps; i += 2) {
            step(std::true_type(), st0, i);
            if (i + 1 < steps) step(std::true_type(), st1, i + 1);
        }
        w0 = w1;
    }
    // o in OUT_UNITs
    const float out_unit = vref * OUT_UNIT;
    const int n_cuts = (rq.units + len - 1) / len;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int row = row0 + 16 * n + c;
        if (row >= rows) continue;
        const float back = -BIAS * ps[n];
        const float sum = rq.too_long ? __builtin_nanf("") : l[n] * OUT_UNIT;
        const size_t at = (size_t)((h * rq.groups + rg) * n_cuts + cut) * a.part_rows + (row - rg * RW);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            f32x4_t v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(o[n][d][e], UNIT, back) * out_unit;
            *reinterpret_cast<f32x4_t *>(a.part + at * D + 16 * d + 4 * g) = v;
        }
        if (g == 0) *reinterpret_cast<f32x2_t *>(a.part_ml + 2 * at) = f32x2_t{m[n], sum};
    }
}

// kv_prefix_rows_kernel's variant for more than 16 rows (M * G) to a KV head.
struct PrefixShape {
    int NR, WAVES;  // row tiles of a wave, waves
};
// One row tile a wave, three workgroups a CU, for heads of 128 up to 192 rows
// (8 heads behind 4096 / 32768 tokens: 64 rows 27.3 / 41.4 us against 30.0 / 47.5
// of two tiles, 128 rows 35.4 / 57.8 against 38.9 / 60.6; behind 32768 192 rows
// 68.3 against 72.0, 256 rows 79.8 against 74.5, 512 rows 129 against 110).  Heads
// of 256 have registers for one tile: four waves up to 64 rows, which is what
// they hold (49.7 us against 50.4 of eight), eight above (4 heads, 96 rows 54.3
// against 56.8, 512 rows 113 against 128).  The requests' kernel, a wave for all
// rows of a step, takes 22.8 us for 24 rows behind 4096 tokens (here 18.8), 25.9
// for 32 behind 8192 (21.6), 47.7 for 64 behind 32768; heads of 64, 32 rows
// 19.4 (18.5).
constexpr PrefixShape prefix_shape(int D, int64_t rows) {
    if (D == 256) return {1, rows <= 64 ? 4 : 8};
    return {D == 128 && rows <= 192 ? 1 : 2, 4};
}
// Up to 16 rows the prefix lies on the requests' line, in one launch (4
// requests, 8 heads of 128 behind 8192 tokens 17.4 us against 21.2 in a launch
// of its own, 32768 tokens 25.3 against 38.7).
constexpr bool on_one_line(int64_t rows) { return rows <= 16; }

// The requests' variant, for the rows that one of them can have.
Shape own_shape(int64_t D, int64_t M, int64_t max_q, int64_t G) { return shape_of((int)D, (max_q < M ? max_q : M) * G); }

template <bool E4M3, int D, int NR, int RS, KvMode MODE, int WAVES = 4>
void run_line(const KvAttnArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((kv_attn_kernel<E4M3, D, NR, RS, WAVES, MODE>), dim3((unsigned)a.slots), dim3(WAVES * 64), 0, s, a);
}

// Waves of a workgroup of the requests' that joins the prefix's segments, for
// heads of 64 and 128: eight for one row tile, and where no CU gets a second
// workgroup (8 heads of 128 behind 2048 tokens, 4 requests of 32 drafts and 1000
// tokens 61.7 us against 72.6 of four, 16 of 16 and 700 behind 20011 120 against
// 124); else four (64 requests of 32 rows and 300 tokens behind 8192 99 us
// against 111, 64 of 64 rows 167 against 181).
constexpr int last_waves(const Shape &v, int64_t starts) { return v.NR == 1 || starts <= 256 ? 8 : 4; }

// the requests' own tokens
template <bool E4M3, int D, KvMode MODE, int WAVES>
void pick_own(const KvAttnArgs &a, const Shape &v, hipStream_t s) {
    if constexpr (D == 256)
        v.RS == 1 ? run_line<E4M3, D, 1, 1, MODE>(a, s) : v.RS == 2 ? run_line<E4M3, D, 1, 2, MODE>(a, s) : run_line<E4M3, D, 1, 4, MODE>(a, s);
    else if (v.NR == 1)
        run_line<E4M3, D, 1, 1, MODE, MODE == KV_LAST ? 8 : 4>(a, s);
    else
        v.RS == 1 ? run_line<E4M3, D, 2, 1, MODE, WAVES>(a, s) : v.RS == 2 ? run_line<E4M3, D, 2, 2, MODE, WAVES>(a, s) : run_line<E4M3, D, 2, 4, MODE, WAVES>(a, s);
}

template <bool E4M3, int D, int NR, int WAVES>
void run_rows(const KvAttnArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((kv_prefix_rows_kernel<E4M3, D, NR, WAVES>), dim3((unsigned)a.slots), dim3(WAVES * 64), 0, s, a);
}

template <bool E4M3, int D>
void run(const KvAttnArgs &own, const KvAttnArgs &pre, const KvPrefixPlan &p, hipStream_t s) {
    const Shape v = own_shape(D, own.M, own.max_q, own.G);
    const PrefixShape w = prefix_shape(D, (int64_t)own.M * own.G);
    if (p.both) {
        run_line<E4M3, D, 1, 1, KV_BOTH>(own, s);
    } else {
        if constexpr (D == 256)
            w.WAVES == 4 ? run_rows<E4M3, D, 1, 4>(pre, s) : run_rows<E4M3, D, 1, 8>(pre, s);
        else if (D == 128 && w.NR == 1)
            run_rows<E4M3, D, D == 128 ? 1 : 2, 4>(pre, s);
        else
            run_rows<E4M3, D, 2, 4>(pre, s);
        if (p.last) {
            D == 256 || last_waves(v, p.own_starts) == 4 ? pick_own<E4M3, D, KV_LAST, 4>(own, v, s) : pick_own<E4M3, D, KV_LAST, D == 256 ? 4 : 8>(own, v, s);
            return;
        }
        pick_own<E4M3, D, KV_OWN, 4>(own, v, s);
    }
    KvPrefixJoinArgs j;
    j.own = own;
    j.pre = pre;
    j.own_rw = 16 * v.NR * v.RS;
    j.pre_rw = p.pre_rw;
    j.both = p.both;
    // a wave a join where they fill the GPU, eight below (8 heads of 128, requests of
    // 6000 tokens: 48 requests, 1536 joins, 120 us against 128.5; 16, 512 joins, 66.8
    // against 70.3)
    const int64_t joins = (int64_t)own.R * own.max_q * own.Hq;
    if (joins >= 1024)
        hipLaunchKernelGGL((kv_prefix_join_kernel<D, 1>), dim3((unsigned)((joins + 7) / 8)), dim3(512), 0, s, j);
    else
        hipLaunchKernelGGL((kv_prefix_join_kernel<D, 8>), dim3((unsigned)joins), dim3(512), 0, s, j);
}

}  // namespace

bool kv_prefix_plan(int64_t R, int64_t M, int64_t Hkv, int64_t G, int64_t D, int64_t max_q, int64_t max_len,
                    int64_t max_prefix, KvPrefixPlan *p) {
    M = M > 0 ? M : 1;
    const int64_t rows = (max_q < M ? max_q : M) * G, all = M * G, steps = (max_prefix + KV_STEP - 1) / KV_STEP;
    const Shape v = own_shape(D, M, max_q, G);
    const PrefixShape w = prefix_shape((int)D, all);
    p->both = on_one_line(all);
    const int64_t RW = 16 * v.NR * v.RS, PW = p->both ? RW : 16 * w.NR * w.WAVES;
    const int64_t groups = (rows + RW - 1) / RW, pgroups = (all + PW - 1) / PW, units = (max_len + KV_STEP - 1) / KV_STEP + 1;
    // the requests' line
    KvAttnPlan &o = p->own;
    // (on one line, cut on every start, only the starts of work count: of no more requests than rows)
    const int64_t starts = p->both ? Hkv * ((R < M ? R : M) * groups + pgroups) : R * Hkv * groups;
    int64_t most = R * Hkv * groups * units + (p->both ? Hkv * pgroups * (steps + 1) : 0);
    if (most >= (int64_t(1) << 31) - 65536) return false;
    p->pre_rw = (int)PW;
    o.groups = (int)groups;
    o.whole = false;
    o.slots = 256 * (v.NR == 1 && D <= 128 ? 3 : 2);
    // On one line a workgroup a CU, or as many more as leave four for each start,
    // then two, and a cut falls on every start: fewer segments, and less to join (4
    // requests, 8 heads of 128 behind 8192 tokens 17.4 us against 19.8 of three a
    // CU, 131072 53.5 against 58.4; 12 requests of 16 heads behind 8192 22 against 31
    // of equal runs over all starts, 16 of 32 heads 39 against 48).
    if (p->both) o.slots = (int)(starts <= 64 ? 256 : starts <= 128 ? 512 : 2 * starts > o.slots ? 2 * starts : o.slots);
    o.min_run = 4 / v.RS;
    o.part_rows = (int)(p->both ? 16 : rows < RW ? rows : RW);
    // Else a cut on every start up to one a CU (32 requests of up to 6000 tokens, 8
    // heads of 128: 75 us against 80 of equal runs, of 8 drafts and 2000 86 against
    // 101, heads of 256 92 against 101); above, lengths that differ make parts that
    // do (48 of up to 16000: 171 against 159, 512 of up to 3000 385 against 351).
    o.aligned = p->both || starts <= 256;
    if (!o.aligned) o.slots *= 2;
    o.part_slots = o.slots + (o.aligned ? 0 : starts);
    o.head_bytes = PART_HEAD;
    p->own_starts = (int)starts;
    // the prefix's: parts of at least 3 steps, as many as cost least: rounds of
    // workgroups, each of its steps and of about 12 more of first loads and
    // last sums (6 or 20 made no difference).  Requests that are not cut join the
    // prefix's segments themselves, a launch and a pass over segments less,
    // where contexts are short, or many requests of one row tile fill the GPU:
    // about two steps for each segment of a wave, against 28.
    // Measured, 8 heads of 128 behind 2048 tokens, this against a line of the
    // requests' own and a join: 32 requests of 40 tokens 20.1 us against 30.6,
    // 48 of 1000 39.8 against 49.1, 48 of 4000 86.8 against 95, 48 of 8192 158
    // against 151, 256 of 40 97 against 86; 16 of 16 drafts and 500 tokens 51.6
    // against 60.9, 2000 80.8 against 72.4; 8 of 300, heads of 256, behind
    // 131072 tokens (128 segments) 55 us against 25.
    KvAttnPlan &q = p->pre;
    const int64_t pairs = Hkv * pgroups, fit = 256 * (w.NR == 1 && D == 128 ? 3 : 8 / w.WAVES);
    if (pairs * (steps + 1) >= (int64_t(1) << 31) - 65536) return false;
    const int split = (D <= 128 ? last_waves(v, starts) : 4) / v.RS;  // waves that share a request's segments
    const bool whole = !p->both && starts <= 1024 && (max_len <= 1024 || (v.NR == 1 && D <= 128 && starts >= 128 && max_len <= 4096));
    const int64_t longest = steps / 3 > 1 ? steps / 3 : 1, upto = longest < 4 * fit / pairs ? longest : 4 * fit / pairs;
    int64_t best = 1;
    double least = 1e30;
    p->last = false;
    // On one line there are none to choose.  Of numbers with the same rounds and the
    // same steps the first costs least, so the others are passed over, from the number
    // on below which no two have the same steps (one head, 24 rows behind 131072
    // tokens: 1 us on the host against 6 of trying all).
    for (int64_t k = 1, end = p->both ? 0 : upto > 1 ? upto : 1; k <= end;) {
        const int64_t rounds = (pairs * k + fit - 1) / fit, each = (steps + k - 1) / k;
        const double cost = (double)rounds * ((double)each + 12.0) + (double)(Hkv * all * k * D) * 8.0 / 5e6;
        const double fold = 2.0 + 2.0 * (double)k / split;
        const bool last = whole && fold < 28.0;
        if (cost + (last ? fold : 28.0) < least) {
            least = cost + (last ? fold : 28.0);
            best = k;
            p->last = last;
        }
        int64_t same = k;
        if (k * k > steps) {
            same = rounds * fit / pairs;
            if (each > 1 && (steps - 1) / (each - 1) < same) same = (steps - 1) / (each - 1);
        }
        k = same + 1;
    }
    p->cuts = (int)best;
    q.groups = (int)pgroups;
    q.whole = false;
    q.slots = (int)(p->both ? 0 : pairs * best);
    q.min_run = 1;
    q.part_rows = (int)(all < PW ? all : PW);
    q.aligned = true;
    q.part_slots = q.slots;
    q.head_bytes = p->both ? 0 : PART_HEAD;
    if (p->last) {
        o.slots = (int)starts;  // a workgroup for each (request, head, row group)
        o.part_slots = o.head_bytes = 0;
    }
    const auto bytes = [&](const KvAttnPlan &l) { return (size_t)l.part_slots * (size_t)l.part_rows * (size_t)(D + 2) * 4; };
    const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    p->own_part = up((size_t)(o.head_bytes + q.head_bytes));
    p->pre_part = p->own_part + up(bytes(o));
    p->bytes = p->pre_part + up(bytes(q));
    return q.part_slots < (int64_t(1) << 31) - 65536 && o.part_slots < (int64_t(1) << 31) - 65536;
}

hipError_t launch_kv_prefix_attention(const KvAttnArgs &own, const KvAttnArgs &pre, const KvPrefixPlan &p, int D, bool e4m3,
                                      hipStream_t s) {
    if (e4m3)
        D == 64 ? run<true, 64>(own, pre, p, s) : D == 128 ? run<true, 128>(own, pre, p, s) : run<true, 256>(own, pre, p, s);
    else
        D == 64 ? run<false, 64>(own, pre, p, s) : D == 128 ? run<false, 128>(own, pre, p, s) : run<false, 256>(own, pre, p, s);
    return hipGetLastError();
}

}  // namespace qg
