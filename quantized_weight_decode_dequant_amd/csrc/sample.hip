// The next tokens from the output head's logits: temperature, top-k, top-p,
// min-p and a given uniform number for each row, by inversion.
//
//   w_i = exp((x_i - max) / T)
//   top-k: the first k tokens by (logit down, token up)
//   top-p: of those, the ones whose mass before them is < p * (top-k's mass)
//   min-p: of those, the ones with w_i >= min_p (the largest has w = 1)
//   token = the first, in order of tokens, whose running sum of kept w passes
//           u * (their mass)
//
// A token hangs on where u falls among up to 2^20 borders, so weights and sums
// have to be far better than fp32's: w is computed in fp64 (relative error
// below 2^-47) and rounded to multiples of 2^-42; sums of these are exact
// integers, the same in any order, so atomics may make them.
//
// Filters need no sort.  Tokens are binned by how far they lie below the row's
// largest logit (128 bins to an octave), with counts and masses of the bins; a
// filter's border lies in one bin (or a few: top-p's under top-k, whose mass
// is known up to a part of a bin).  The bins above are kept whole, the tokens
// of the border's bins are listed, and among these a radix descent over their
// logits finds the border.
//
// Kernels of a workgroup for each chunk of 4096 tokens, or for each row:
//   sample_top    (chunk) its waves' largest logits
//   sample_bins   (chunk) counts and masses by bins, or the kept mass
//   sample_find   (row)   the borders' bins; the token of a row without them
//   sample_list   (chunk) its kept mass, and its part of the list
//   sample_pick   (row)   the borders and the token
// Where few workgroups run, sample_list finds the borders' bins in each of them
// instead of a launch by itself (one row 21.7 us against 23.4); without top-k
// and top-p nothing follows sample_find.  One launch each, rather than a row's
// last workgroup going on: the fences that this takes cost 462 us where the
// kernel's work is 30 (192 rows; one row 51 us against 45, both untuned).
//
// One row of 151936, top-k 50, takes 3.1 + 4.4 + 6.7 + 8.0 us, all latency: launches,
// settings, logits, atomics in turn.  16 fp32 rows, top-p alone, 3.8 + 9.0 + 9.8 +
// 11.9. 192 bf16 rows, each with settings of its own, 12.4 (4.7 TB/s) + 25.4 (the
// vector unit: some 33 instructions a token where masses are asked for, most of them
// the weight's) + 4.8 + 13.9 + 16.5.
#include <type_traits>

#include "sample.h"

namespace qg {

namespace {

typedef unsigned long long u64;

constexpr int TH = SAMPLE_THREADS, W = TH / 64, E = SAMPLE_PER_THREAD, NB = SAMPLE_BINS;
constexpr float NEG_INF = -__builtin_inff();
constexpr double UNIT = 0x1p42;  // of masses
// Top-k up to which top-p's border comes from the list alone: so many that a
// workgroup ranks them at once, most often.  151936 tokens, k = 50: one row 20.5 us
// against 21.4, 192 rows 66 against 82; k = 100: 21.4 either way, 71 against 85; k =
// 200, whose list is narrowed by digits: one row 26.4 against 22.1.
constexpr int BY_LIST = 100;

__device__ __forceinline__ float f32_of(unsigned w) { return __builtin_bit_cast(float, w); }
__device__ __forceinline__ unsigned bits_of(float f) { return __builtin_bit_cast(unsigned, f); }

// n logits from token `at` on; NaN past the row's end
template <bool F32, int n>
__device__ __forceinline__ void load_logits(const void *logits, int64_t row, int at, int V, float (&x)[n]) {
    constexpr int N = F32 || n < 8 ? 4 : 8;  // of one load
    const char *p = (const char *)logits + (row + at) * (F32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < n; i += N) {
        if (at + i + N <= V) {
            constexpr int WORDS = F32 ? 4 : N / 2;
            unsigned w[WORDS];
            __builtin_memcpy(w, p + i * (F32 ? 4 : 2), WORDS * 4);  // rows are aligned to an element only
#pragma unroll
            for (int e = 0; e < WORDS; ++e) {
                const unsigned u = w[e];
                if (F32) {
                    x[i + e] = f32_of(u);
                } else {
                    x[i + 2 * e] = bf16_lo(u);
                    x[i + 2 * e + 1] = bf16_hi(u);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                x[i + e] = __builtin_nanf("");
                if (at + i + e < V) {
                    if (F32)
                        x[i + e] = ((const float *)p)[i + e];
                    else
                        x[i + e] = f32_of((unsigned)((const uint16_t *)p)[i + e] << 16);
                }
            }
        }
    }
}

// What a row asks for.
struct Ask {
    double c;        // log2(e) / T
    double p, minp;  // p >= 1: no top-p; minp <= 0: no min-p
    int k;           // 0: no top-k
    bool greedy;     // the largest logit
    __device__ __forceinline__ bool filters() const { return k > 0 || p < 1.0; }
    // top-p under so small a top-k that all of top-k's tokens go to the list: no
    // masses by bins, a weight for each listed token instead of each of the row
    __device__ __forceinline__ bool by_list() const { return k > 0 && k <= BY_LIST && p < 1.0; }
};

__device__ __forceinline__ Ask ask_of(const SampleArgs &a, int m) {
    Ask q;
    const float T = a.temperature ? a.temperature[m] : 1.f;
    const int k = a.top_k ? a.top_k[m] : 0;
    const float p = a.top_p ? a.top_p[m] : 1.f, minp = a.min_p ? a.min_p[m] : 0.f;
    q.greedy = !(T > 0.f) || k == 1;
    q.c = 1.44269504088896340736 / (double)T;
    q.k = k > 0 && k < a.V ? k : 0;
    q.p = p < 1.f ? fmax((double)p, 0.0) : 1.0;  // (NaN: off; its products become whole numbers, so none is negative)
    q.minp = minp > 0.f ? fmin((double)minp, 1.0) : 0.0;
    return q;
}

// 2^-(j / 32), for weights
__device__ __forceinline__ void make_powers(double *pow) {
    if (threadIdx.x < 32) pow[threadIdx.x] = exp2(-(double)threadIdx.x * 0.03125);
}

// Logits as a row sees them, relative to its largest: `top`, what makes them
// finite where that is infinite, and from which distance on (in halves, which
// cannot overflow) a weight is below 2^-44, a quarter of its unit: such tokens, NaN
// and -infinity among them, are dead, they are never drawn and do not count.  (Those
// up to 2^-43 round to a mass of 0: never drawn either.)
struct Scale {
    float top, half_top, reach;
    bool infinite;
    __device__ __forceinline__ float distance(float x) const { return fmaf(-0.5f, x, half_top); }
    __device__ __forceinline__ bool dead(float d) const { return !(d <= reach); }
    template <int n>
    __device__ __forceinline__ void settle(float (&x)[n]) const {
        if (infinite) {
#pragma unroll
            for (int e = 0; e < n; ++e) x[e] = x[e] == -NEG_INF ? 0.f : NEG_INF;
        }
    }
};

__device__ __forceinline__ Scale scale_of(float top, const Ask &q) {
    Scale s;
    s.infinite = top == -NEG_INF;
    s.top = s.infinite ? 0.f : top;
    s.half_top = 0.5f * s.top;
    s.reach = fminf((float)(22.0 / q.c), 3.4e38f);
    return s;
}

// exp((x - top) / T): 2^-t by t = (32 n + j) / 32 + rest, |rest| <= 1/64, the
// rest's power by its series to the fifth order (2e-15).  0 of NaN.
__device__ __forceinline__ double weight(float x, float top, double c, const double *pow) {
    const double t = fmin(((double)top - (double)x) * c, 1100.0);
    constexpr double MAGIC = 0x1.8p52, S = -0.69314718055994530942 / 32;
    const double y = fma(t, 32.0, MAGIC);
    const int n = (int)(unsigned)__builtin_bit_cast(u64, y);
    const double r = fma(t, 32.0, -(y - MAGIC));
    double q = fma(r, S * S * S * S * S / 120, S * S * S * S / 24);
    q = fma(r, q, S * S * S / 6);
    q = fma(r, q, S * S / 2);
    q = fma(r, q, S);
    q = fma(r, q, 1.0);
    return ldexp(pow[n & 31] * q, -(n >> 5));
}

// in units of 2^-42, to the nearest
__device__ __forceinline__ u64 mass_of(double w) {
    return __builtin_bit_cast(u64, fma(w, UNIT, 0x1p52)) & 0xFFFFFFFFFFFFFull;
}

// Larger keys for larger logits; one key for both zeros.
__device__ __forceinline__ unsigned key_of(float x) {
    const unsigned u = bits_of(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float logit_of(unsigned key) { return f32_of(key & 0x80000000u ? key ^ 0x80000000u : ~key); }

// 128 bins to an octave of the distance from the top, from 1/32 of halves on.
__device__ __forceinline__ int bin_of(float d) { return min(max((int)(bits_of(d) >> 16) - ((127 - 5) << 7), 0), NB - 1); }

// v of the lane that a DPP control names; 0 where it names none.
template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned from_lane(unsigned v) {
    return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 from_lane(u64 v) {
    return (u64)from_lane<CTRL, ROWS>((unsigned)v) | ((u64)from_lane<CTRL, ROWS>((unsigned)(v >> 32)) << 32);
}

// Sum over the wave's lanes up to this one: within rows of 16 lanes (shifts by
// 1, 2, 4, 8), then each row's last lane into the rows behind.
template <typename T>
__device__ __forceinline__ T scan_wave(T v) {
    v += from_lane<0x111, 0xF>(v);
    v += from_lane<0x112, 0xF>(v);
    v += from_lane<0x114, 0xF>(v);
    v += from_lane<0x118, 0xF>(v);
    v += from_lane<0x142, 0xA>(v);
    v += from_lane<0x143, 0xC>(v);
    return v;
}

// Sum over the workgroup's threads before this one, and over all.
template <typename T>
__device__ __forceinline__ T scan_before(T v, T *waves, T &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const T upto = scan_wave(v);
    __syncthreads();
    if (lane == 63) waves[wave] = upto;
    __syncthreads();
    T before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const T u = waves[w];
        if (w < wave) before += u;
        total += u;
    }
    return before + upto - v;
}

__device__ __forceinline__ u64 sum_all(u64 v, u64 *waves) {
    u64 total;
    scan_before(v, waves, total);
    return total;
}

template <int CTRL>
__device__ __forceinline__ float max_lane(float v) {
    const int u = (int)bits_of(v);
    return fmaxf(v, f32_of((unsigned)__builtin_amdgcn_update_dpp(u, u, CTRL, 0xF, 0xF, false)));
}

// The wave's largest, in its last lane.
__device__ __forceinline__ float max_wave(float v) {
    v = max_lane<0x111>(v);
    v = max_lane<0x112>(v);
    v = max_lane<0x114>(v);
    v = max_lane<0x118>(v);
    v = max_lane<0x142>(v);
    return max_lane<0x143>(v);
}

__device__ __forceinline__ float max_all(float v, float *waves) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = max_wave(v);
    __syncthreads();
    if (lane == 63) waves[wave] = v;
    __syncthreads();
    v = waves[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v = fmaxf(v, waves[w]);
    return v;
}

// A row's largest logit, from its chunks'.
__device__ __forceinline__ float top_of(const SampleArgs &a, int m, float &mine, float *waves) {
    mine = NEG_INF;
    if ((int)threadIdx.x < a.chunks) {
        const f32x4_t t = *reinterpret_cast<const f32x4_t *>(a.tops + ((size_t)m * a.chunks + threadIdx.x) * SAMPLE_SUBS);
        mine = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
    }
    return max_all(mine, waves);
}

// ------------------------------------------------------------------ the chunks' largest
template <bool F32>
__global__ void __launch_bounds__(TH) sample_top_kernel(SampleArgs a) {
    const int c = blockIdx.x % a.chunks, m = blockIdx.x / a.chunks, tid = threadIdx.x;
    float x[E];
    load_logits<F32>(a.logits, (int64_t)m * a.stride, c * SAMPLE_CHUNK + tid * E, a.V, x);
    if (a.top_k || a.top_p) {
        for (int i = c * TH + tid; i < NB; i += a.chunks * TH) {
            a.masses[(size_t)m * NB + i] = 0;
            a.counts[(size_t)m * NB + i] = 0;
        }
    }
    if (c == 0 && tid == 0) a.rows[m].listed = 0;
    float top = NEG_INF;
#pragma unroll
    for (int e = 0; e < E; ++e) top = fmaxf(top, x[e]);  // (past NaN)
    top = f32_of((unsigned)__builtin_amdgcn_readlane((int)bits_of(max_wave(top)), 63));
    int at = -1;
#pragma unroll
    for (int e = E - 1; e >= 0; --e)
        if (x[e] == top) at = c * SAMPLE_CHUNK + tid * E + e;
    const unsigned long long has = __ballot(at >= 0);
    if ((tid & 63) == (has ? (int)__builtin_ctzll(has) : 0)) {
        const size_t part = ((size_t)m * a.chunks + c) * SAMPLE_SUBS + tid / 64;
        a.tops[part] = top;
        a.top_at[part] = at;
    }
}

// ------------------------------------------------------------------ counts and masses by bins
template <bool F32>
__global__ void __launch_bounds__(TH) sample_bins_kernel(SampleArgs a) {
    __shared__ double pow[32];
    __shared__ u64 waves[TH / 64];
    __shared__ u64 masses[NB];
    __shared__ unsigned counts[NB];
    const int c = blockIdx.x % a.chunks, m = blockIdx.x / a.chunks, tid = threadIdx.x;
    const Ask q = ask_of(a, m);
    if (!a.few && q.greedy) return;
    float x[E], mine;
    load_logits<F32>(a.logits, (int64_t)m * a.stride, c * SAMPLE_CHUNK + tid * E, a.V, x);
    make_powers(pow);
#pragma unroll
    for (int i = 0; i < NB / TH; ++i) {
        masses[i * TH + tid] = 0;
        counts[i * TH + tid] = 0;
    }
    if (q.greedy) return;
    const Scale t = scale_of(top_of(a, m, mine, (float *)waves), q);
    t.settle(x);
    if (!q.filters()) {
        u64 sum = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (t.dead(t.distance(x[e]))) continue;
            const double v = weight(x[e], t.top, q.c, pow);
            sum += v >= q.minp ? mass_of(v) : 0;
        }
        sum = scan_wave(sum);
        if ((tid & 63) == 63) a.kept[((size_t)m * a.chunks + c) * SAMPLE_SUBS + tid / 64] = sum;
        return;
    }
    const bool by_mass = q.p < 1.0 && !q.by_list();
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float d = t.distance(x[e]);
        if (!t.dead(d)) {
            const int b = bin_of(d);
            if (q.k > 0) atomicAdd(&counts[b], 1u);
            if (by_mass) atomicAdd(&masses[b], mass_of(weight(x[e], t.top, q.c, pow)));
        }
    }
    __syncthreads();
    unsigned n[NB / TH];
    u64 w[NB / TH];
#pragma unroll
    for (int i = 0; i < NB / TH; ++i) {
        n[i] = counts[i * TH + tid];
        w[i] = masses[i * TH + tid];
    }
#pragma unroll
    for (int i = 0; i < NB / TH; ++i) {
        if (n[i]) atomicAdd(&a.counts[(size_t)m * NB + i * TH + tid], n[i]);
        if (w[i]) atomicAdd(&a.masses[(size_t)m * NB + i * TH + tid], w[i]);
    }
}

// ------------------------------------------------------------------ by rows
// What a row's workgroup keeps in LDS.
constexpr int DIGITS = TH;  // of a level of the descent
struct Shared {
    double pow[32];
    union {
        u64 wave64[W];
        unsigned wave32[W];
        float wavef[W];
    };
    u64 found64[2];
    unsigned found32[4];
    u64 mass[TH * SAMPLE_SUBS];  // by digit, then by part of a chunk
    unsigned count[TH * SAMPLE_SUBS];
};
constexpr int SUB = SAMPLE_CHUNK / SAMPLE_SUBS;  // tokens of a part

// A row's cut in terms of its undecided tokens: those of larger keys are kept,
// and of this key the first `ties` as far as `token`.
struct Cut {
    unsigned key, token, ties;
};

// Whether a filter's border lies in this bin.
__device__ __forceinline__ bool undecided(const SampleRow &r, int b) {
    return (b >= r.p_lo && b <= r.p_hi) || b == r.k_bin;
}

// The token, from the kept masses of the chunks' parts (`mine`: of chunk tid)
// and, where there are filters (`row`), their numbers of the cut key's tokens
// (`ties`; `ties_before`: before chunk tid).
template <bool F32>
__device__ __forceinline__ void pick(const SampleArgs &a, int m, const Ask &q, const Scale &s, const u64 (&mine)[SAMPLE_SUBS], const SampleRow *row,
                                     Cut cut, const unsigned *ties, unsigned ties_before, Shared &sh) {
    constexpr int PE = SUB / TH;
    const int tid = threadIdx.x;
    u64 total, sum = 0;
#pragma unroll
    for (int i = 0; i < SAMPLE_SUBS; ++i) sum += mine[i];
    u64 before = scan_before(sum, sh.wave64, total);
    if (total == 0) {  // (only -infinities and NaN)
        if (tid == 0) {
            a.tokens[m] = -1;
            if (a.logprobs) a.logprobs[m] = __builtin_nanf("");
        }
        return;
    }
    const double u = (double)a.u[m];
    u64 r = u > 0.0 ? (u64)(fmin(u, 1.0) * (double)total) : 0;
    r = r < total ? r : total - 1;
    const bool by_ties = row && ties;
#pragma unroll
    for (int i = 0; i < SAMPLE_SUBS; ++i) {
        if (mine[i] > 0 && r >= before && r - before < mine[i]) {
            sh.found32[0] = (unsigned)(tid * SAMPLE_SUBS + i);
            sh.found32[1] = ties_before;
            sh.found64[0] = r - before;
        }
        before += mine[i];
        if (by_ties) ties_before += ties[i];
    }
    __syncthreads();
    const int at = (int)sh.found32[0] * SUB + tid * PE;
    r = sh.found64[0];
    float x[PE];
    load_logits<F32>(a.logits, (int64_t)m * a.stride, at, a.V, x);
    s.settle(x);
    unsigned place = 0;  // of this thread's first token of the cut key among all
    if (by_ties) {
        unsigned n = 0, all;
#pragma unroll
        for (int e = 0; e < PE; ++e) {
            const float d = s.distance(x[e]);
            n += !s.dead(d) && key_of(x[e]) == cut.key && undecided(*row, bin_of(d));
        }
        place = sh.found32[1];
        place += scan_before(n, sh.wave32, all);
    }
    u64 w[PE];
    double v[PE];
    sum = 0;
#pragma unroll
    for (int e = 0; e < PE; ++e) {
        v[e] = weight(x[e], s.top, q.c, sh.pow);
        const float d = s.distance(x[e]);
        bool keep = v[e] >= q.minp && !s.dead(d);
        if (row && keep) {
            const int b = bin_of(d);
            const unsigned key = key_of(x[e]);
            if (undecided(*row, b)) {
                const bool tie = key == cut.key;
                keep = key > cut.key || (tie && (unsigned)(at + e) <= cut.token && place < cut.ties);
                place += by_ties && tie;
            } else {
                keep = b < row->full;
            }
        }
        w[e] = keep ? mass_of(v[e]) : 0;
        sum += w[e];
    }
    u64 from = scan_before(sum, sh.wave64, sum);
    int hit = -1;
    double share = 0.0;
#pragma unroll
    for (int e = 0; e < PE; ++e) {
        if (w[e] > 0 && r >= from && r - from < w[e]) {
            hit = at + e;
            share = v[e];
        }
        from += w[e];
    }
    if (hit >= 0) {
        a.tokens[m] = hit;
        if (a.logprobs) a.logprobs[m] = (float)log(share / ((double)total * (1.0 / UNIT)));
    }
}

// The kept masses of chunk tid's parts.
__device__ __forceinline__ void load_kept(const SampleArgs &a, int m, bool there, u64 (&kept)[SAMPLE_SUBS]) {
#pragma unroll
    for (int i = 0; i < SAMPLE_SUBS; ++i)
        kept[i] = there && (int)threadIdx.x < a.chunks ? a.kept[((size_t)m * a.chunks + threadIdx.x) * SAMPLE_SUBS + i] : 0;
}

// Finds the bins of a row's borders, by the whole workgroup; false where there
// are none to find: the row's token is its largest, or hangs on its kept masses
// alone.
__device__ __forceinline__ bool find_borders(const SampleArgs &a, int m, const Ask &q, float top, SampleRow &r, Shared &sh) {
    constexpr int PER = NB / TH;  // consecutive bins a thread
    const int tid = threadIdx.x;
    if (q.greedy || !q.filters() || top == NEG_INF) return false;
    u64 mass[PER], sum = 0;
    unsigned count[PER], n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        mass[i] = a.masses[(size_t)m * NB + tid * PER + i];
        count[i] = a.counts[(size_t)m * NB + tid * PER + i];
        sum += mass[i];
        n += count[i];
    }
    u64 total;
    unsigned tokens;
    const u64 mass_before = scan_before(sum, sh.wave64, total);
    const unsigned count_before = scan_before(n, sh.wave32, tokens);
    if (tid == 0) {
        sh.found64[0] = sh.found64[1] = total;   // mass before top-k's bin, and with it
        sh.found32[2] = sh.found32[3] = NB - 1;  // top-p's bins
    }
    __syncthreads();
    const bool by_k = q.k > 0 && (unsigned)q.k < tokens;  // (of those that are not dead)
    if (by_k) {
        u64 s = mass_before;
        unsigned k = count_before;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (k < (unsigned)q.k && k + count[i] >= (unsigned)q.k) {
                sh.found32[0] = tid * PER + i;
                sh.found32[1] = (unsigned)q.k - k;
                sh.found64[0] = s;
                sh.found64[1] = s + mass[i];
            }
            k += count[i];
            s += mass[i];
        }
    }
    __syncthreads();
    const u64 lo = sh.found64[0], hi = sh.found64[1];  // top-k's mass lies between
    const bool by_p = q.p < 1.0;
    r.k_bin = by_k ? (int)sh.found32[0] : -1;
    r.k_left = by_k ? sh.found32[1] : 0;
    __syncthreads();
    if (q.by_list()) {
        if (tid == 0) {
            sh.found32[2] = 0;
            sh.found32[3] = by_k ? (unsigned)r.k_bin : NB - 1;
        }
    } else if (by_p) {
        const u64 want_lo = max((u64)ceil(q.p * (double)lo), (u64)1), want_hi = max((u64)ceil(q.p * (double)hi), (u64)1);
        u64 s = mass_before;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (s < want_lo && s + mass[i] >= want_lo) {
                sh.found32[2] = tid * PER + i;
                sh.found64[0] = s;
            }
            if (s < want_hi && s + mass[i] >= want_hi) sh.found32[3] = tid * PER + i;
            s += mass[i];
        }
    }
    __syncthreads();
    r.done = 0;
    r.listed = 0;
    r.top = top;
    r.p_lo = by_p ? (int)sh.found32[2] : NB;
    r.p_hi = by_p ? (int)sh.found32[3] : -1;
    r.full = by_p ? r.p_lo : by_k ? r.k_bin : NB;
    r.p_mass = sh.found64[0];
    r.k_mass = lo;
    r.mass = total;
    return true;
}

// A row without borders: its token.
template <bool F32>
__device__ __forceinline__ void finish_row(const SampleArgs &a, int m, const Ask &q, float top, float mine, Shared &sh) {
    const int tid = threadIdx.x;
    const bool none = top == NEG_INF;  // of finite or infinite logits
    if (tid == 0) {
        sh.found32[0] = 0x7FFFFFFF;
        a.rows[m].done = 1;
    }
    __syncthreads();
    if (!q.greedy) {
        u64 kept[SAMPLE_SUBS];
        load_kept(a, m, !none, kept);
        pick<F32>(a, m, q, scale_of(top, q), kept, nullptr, Cut{0, 0, 0}, nullptr, 0, sh);
        return;
    }
    if (tid < a.chunks && mine == top) {
#pragma unroll
        for (int i = SAMPLE_SUBS - 1; i >= 0; --i) {
            const size_t part = ((size_t)m * a.chunks + tid) * SAMPLE_SUBS + i;
            if (a.tops[part] == top && a.top_at[part] >= 0) atomicMin(&sh.found32[0], (unsigned)a.top_at[part]);
        }
    }
    __syncthreads();
    if (tid == 0) {
        a.tokens[m] = none ? -1 : (int)sh.found32[0];
        if (a.logprobs) a.logprobs[m] = none ? __builtin_nanf("") : 0.f;
    }
}

template <bool F32>
__global__ void __launch_bounds__(TH) sample_find_kernel(SampleArgs a) {
    __shared__ Shared sh;
    const int m = blockIdx.x;
    const Ask q = ask_of(a, m);
    make_powers(sh.pow);
    float mine;
    const float top = top_of(a, m, mine, sh.wavef);
    SampleRow r;
    if (!find_borders(a, m, q, top, r, sh)) {
        finish_row<F32>(a, m, q, top, mine, sh);
    } else if (threadIdx.x == 0) {
        a.rows[m] = r;
    }
}

// ------------------------------------------------------------------ the list
// FIND: the borders' bins are found by each of a row's workgroups for itself,
// and left for the next kernel by the first, which also ends rows without.
template <bool F32, bool FIND>
__global__ void __launch_bounds__(TH) sample_list_kernel(SampleArgs a) {
    __shared__ Shared sh;
    __shared__ unsigned first;
    const int c = blockIdx.x % a.chunks, m = blockIdx.x / a.chunks, tid = threadIdx.x;
    SampleRow r;
    Ask q;
    float x[E], top, mine;
    if (FIND) {
        q = ask_of(a, m);
        load_logits<F32>(a.logits, (int64_t)m * a.stride, c * SAMPLE_CHUNK + tid * E, a.V, x);
        top = top_of(a, m, mine, sh.wavef);
    } else {
        r = a.rows[m];
        if (r.done) return;
        q = ask_of(a, m);
        top = r.top;
        // a wave, or a workgroup, whose largest lies behind all borders has nothing
        // to read
        const Scale t = scale_of(top, q);
        const size_t part = ((size_t)m * a.chunks + c) * SAMPLE_SUBS;
        const int last = max(max(r.p_hi, r.k_bin), r.full - 1);
        bool any = false, mine_any = false;
#pragma unroll
        for (int i = 0; i < SAMPLE_SUBS; ++i) {
            const float d = t.infinite ? (a.tops[part + i] == top ? 0.f : -NEG_INF) : t.distance(a.tops[part + i]);
            const bool has = !t.dead(d) && bin_of(d) <= last;
            any |= has;
            if (i == __builtin_amdgcn_readfirstlane(tid / 64)) mine_any = has;
        }
        if (!any) {
            if (tid < SAMPLE_SUBS) a.kept[part + tid] = 0;
            return;
        }
        if (mine_any) {
            load_logits<F32>(a.logits, (int64_t)m * a.stride, c * SAMPLE_CHUNK + tid * E, a.V, x);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = __builtin_nanf("");
        }
    }
    make_powers(sh.pow);
    __syncthreads();
    if (FIND) {
        if (!find_borders(a, m, q, top, r, sh)) {
            if (c == 0) finish_row<F32>(a, m, q, top, mine, sh);
            return;
        }
        if (c == 0 && tid == 0) {
            SampleRow *to = a.rows + m;  // (its count of the list is the others' already)
            to->done = 0;
            to->top = top;
            to->full = r.full;
            to->p_lo = r.p_lo;
            to->p_hi = r.p_hi;
            to->k_bin = r.k_bin;
            to->k_left = r.k_left;
            to->p_mass = r.p_mass;
            to->k_mass = r.k_mass;
            to->mass = r.mass;
        }
    }
    const Scale t = scale_of(top, q);
    t.settle(x);
    u64 sum = 0;
    unsigned open = 0, n = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float d = t.distance(x[e]);
        if (t.dead(d)) continue;
        const int b = bin_of(d);
        if (b < r.full) {
            const double v = weight(x[e], t.top, q.c, sh.pow);
            sum += v >= q.minp ? mass_of(v) : 0;
        } else if (undecided(r, b)) {
            open |= 1u << e;
            ++n;
        }
    }
    sum = scan_wave(sum);
    if ((tid & 63) == 63) a.kept[((size_t)m * a.chunks + c) * SAMPLE_SUBS + tid / 64] = sum;
    unsigned all;
    unsigned place = scan_before(n, sh.wave32, all);
    if (tid == 0) {
        // (chunks come in any order: what is made of the list does not depend on it)
        if (all > 0) first = atomicAdd(&a.rows[m].listed, all);
    }
    if (all == 0) return;
    __syncthreads();
    place += first;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (open >> e & 1) {
            if (place < SAMPLE_LIST) a.lists[(size_t)m * SAMPLE_LIST + place] = u32x2_t{key_of(x[e]), (unsigned)(c * SAMPLE_CHUNK + tid * E + e)};
            ++place;
        }
    }
}

// ------------------------------------------------------------------ the borders, and the token
// So many tokens are taken by rank, each against all others (of 256, that took
// 6 us; a descent takes 5).
constexpr unsigned BRIEF = 128;
static_assert(BRIEF <= TH, "a token a thread");

// Number and mass of the n tokens before `order`; few[] is filled up to a
// multiple of four with tokens that come last.
__device__ __forceinline__ u64 before_of(u64 order, const ulonglong2 *few, unsigned n, unsigned &rank) {
    u64 mass = 0;
    rank = 0;
    for (unsigned j = 0; j < n; j += 4) {
#pragma unroll
        for (unsigned e = 0; e < 4; ++e) {
            const ulonglong2 t = few[j + e];
            rank += t.x > order;
            mass += t.x > order ? t.y : 0;
        }
    }
    return mass;
}

template <bool F32>
__global__ void __launch_bounds__(TH) sample_pick_kernel(SampleArgs a) {
    __shared__ Shared sh;
    __shared__ u32x2_t held[SAMPLE_LIST];
    __shared__ ulonglong2 few[BRIEF + 4];  // a few tokens' order (larger: earlier) and mass
    const int m = blockIdx.x, tid = threadIdx.x;
    const SampleRow r = a.rows[m];
    if (r.done) return;
    const Ask q = ask_of(a, m);
    const u32x2_t *list = a.lists + (size_t)m * SAMPLE_LIST;
    const bool brief = r.listed <= BRIEF;  // a token of the list for each thread
    u32x2_t own = {0u, 0u};
    if (brief) {
        if ((unsigned)tid < r.listed) own = list[tid];
    } else if (r.listed <= SAMPLE_LIST) {
#pragma unroll 8
        for (unsigned i = tid; i < r.listed; i += TH) held[i] = list[i];
    }
    u64 kept[SAMPLE_SUBS];
    load_kept(a, m, true, kept);
    make_powers(sh.pow);
    const Scale t = scale_of(r.top, q);
    __syncthreads();
    const auto mass_at = [&](unsigned key) { return mass_of(weight(logit_of(key), t.top, q.c, sh.pow)); };
    const auto bin_at = [&](unsigned key) { return bin_of(t.distance(logit_of(key))); };

    if (brief) {
        // every token's rank and the mass before it, against all others
        const bool valid = (unsigned)tid < r.listed;
        const double v = valid ? weight(logit_of(own[0]), t.top, q.c, sh.pow) : 0.0;
        const u64 w = mass_of(v), order = ((u64)own[0] << 32) | ~own[1];  // larger: earlier
        const int b = valid ? bin_at(own[0]) : NB;
        if (tid < (int)BRIEF + 4) few[tid] = valid ? ulonglong2{order, w} : ulonglong2{0, 0};
        if (tid == 0) sh.found64[0] = ~0ull;
        const unsigned sooner = (unsigned)__syncthreads_count(b < r.k_bin);  // listed, before top-k's bin
        unsigned rank;
        const u64 before = r.p_mass + before_of(order, few, r.listed, rank);
        bool keep = valid && (r.k_bin < 0 || rank < r.k_left + sooner);
        if (q.p < 1.0) {
            u64 mass = r.mass;  // what top-k keeps
            if (q.by_list())
                mass = sum_all(keep ? w : 0, sh.wave64);
            else if (r.k_bin >= 0)
                mass = r.k_mass + sum_all(keep && b == r.k_bin ? w : 0, sh.wave64);
            keep &= b <= r.p_hi && before < max((u64)ceil(q.p * (double)mass), (u64)1);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < SAMPLE_SUBS; ++i) sh.mass[i * TH + tid] = 0;
        __syncthreads();
        // kept is what comes first, as far as the last of them
        u64 last = keep ? order : ~0ull;
#pragma unroll
        for (int d = 32; d; d >>= 1) last = min(last, (u64)__shfl_xor(last, d));
        if ((tid & 63) == 0) atomicMin(&sh.found64[0], last);
        if (keep && v >= q.minp) atomicAdd(&sh.mass[own[1] / SUB], w);
        __syncthreads();
        last = sh.found64[0];
#pragma unroll
        for (int i = 0; i < SAMPLE_SUBS; ++i) kept[i] += sh.mass[tid * SAMPLE_SUBS + i];
        pick<F32>(a, m, q, t, kept, &r, Cut{(unsigned)(last >> 32), ~(unsigned)last, ~0u}, nullptr, 0, sh);
        return;
    }

    // f(key, bin, token) for each undecided token
    const auto each = [&](auto f) {
        if (r.listed <= SAMPLE_LIST) {
            for (unsigned i = tid; i < r.listed; i += TH) {
                const u32x2_t one = held[i];
                f(one[0], bin_at(one[0]), one[1]);
            }
        } else {  // more than the list holds: from the logits again
            for (int i = tid; i < a.V; i += TH) {
                const int64_t at = (int64_t)m * a.stride + i;
                float x[1] = {F32 ? ((const float *)a.logits)[at] : f32_of((unsigned)((const uint16_t *)a.logits)[at] << 16)};
                t.settle(x);
                const float d = t.distance(x[0]);
                if (!t.dead(d) && undecided(r, bin_of(d))) f(key_of(x[0]), bin_of(d), (unsigned)i);
            }
        }
    };

    // Among the undecided tokens that `in` takes, the largest first: where
    // `want` of them are together (or, by mass, where the mass with them reaches
    // `want`).  Digits of 8 bits, from the first in which keys differ, until
    // a workgroup's threads can take a token each: those by rank and the mass
    // before them.
    const auto descend = [&](auto by_mass, u64 want, auto in) {
        constexpr bool MASS = decltype(by_mass)::value;
        unsigned least = ~0u, most = 0;
        each([&](unsigned key, int b, unsigned) {
            if (in(key, b)) {
                least = min(least, key);
                most = max(most, key);
            }
        });
#pragma unroll
        for (int d = 32; d; d >>= 1) {
            least = min(least, (unsigned)__shfl_xor((int)least, d));
            most = max(most, (unsigned)__shfl_xor((int)most, d));
        }
        __syncthreads();
        if (tid == 0) {
            sh.found32[2] = ~0u;
            sh.found32[3] = 0;
        }
        __syncthreads();
        if ((tid & 63) == 0) {
            atomicMin(&sh.found32[2], least);
            atomicMax(&sh.found32[3], most);
        }
        __syncthreads();
        least = sh.found32[2];
        most = sh.found32[3];
        if (least > most) return Cut{0, ~0u, 0};  // (no such token)
        int bits = least == most ? 0 : 32 - __clz((int)(least ^ most));
        unsigned prefix = bits < 32 ? most >> bits << bits : 0u, here = 0;
        u64 above = 0;
        do {
            const int shift = max(bits - 8, 0);
            sh.mass[tid] = 0;
            sh.count[tid] = 0;
            __syncthreads();
            each([&](unsigned key, int b, unsigned) {
                if (!in(key, b) || (bits < 32 && (key >> bits) != (prefix >> bits))) return;
                const unsigned d = (DIGITS - 1) - ((key >> shift) & ((1u << (bits - shift)) - 1));
                atomicAdd(&sh.count[d], 1u);
                if (MASS) atomicAdd(&sh.mass[d], mass_at(key));
            });
            __syncthreads();
            const unsigned n = sh.count[tid];
            const u64 v = MASS ? sh.mass[tid] : (u64)n;
            u64 total;
            const u64 before = above + scan_before(v, sh.wave64, total);
            if (tid == 0) sh.found32[0] = DIGITS;
            __syncthreads();
            if (before < want && before + v >= want) {
                sh.found32[0] = tid;
                sh.found32[1] = n;
                sh.found64[0] = before;
            }
            __syncthreads();
            const unsigned d = sh.found32[0];
            if (d == DIGITS) return Cut{0, ~0u, 0};  // (not reached: all are kept)
            prefix |= (DIGITS - 1 - d) << shift;
            here = sh.found32[1];
            above = sh.found64[0];
            bits = shift;
            __syncthreads();
        } while (bits > 0 && here > BRIEF);
        if (bits > 0) {
            if (tid == 0) {
                sh.found32[0] = 0;
                sh.found64[0] = ~0ull;
            }
            if (tid < (int)BRIEF + 4) few[tid] = ulonglong2{0, 0};
            __syncthreads();
            each([&](unsigned key, int b, unsigned token) {
                if (!in(key, b) || key >> bits != prefix >> bits) return;
                few[atomicAdd(&sh.found32[0], 1u)] = ulonglong2{((u64)key << 32) | ~token, MASS ? mass_at(key) : 1};
            });
            __syncthreads();
            u64 last = ~0ull;
            if ((unsigned)tid < here) {
                const u64 order = few[tid].x;
                unsigned rank;
                if (above + before_of(order, few, here, rank) < want) last = order;
            }
#pragma unroll
            for (int d = 32; d; d >>= 1) last = min(last, (u64)__shfl_xor(last, d));
            if ((tid & 63) == 0) atomicMin(&sh.found64[0], last);
            __syncthreads();
            last = sh.found64[0];
            return Cut{(unsigned)(last >> 32), ~(unsigned)last, ~0u};
        }
        u64 ties = want - above;
        if (MASS) {
            const u64 w = mass_at(prefix);
            ties = w > 0 ? (ties + w - 1) / w : here;
        }
        return Cut{prefix, ~0u, ties < here ? (unsigned)ties : here};
    };

    __syncthreads();
    Cut cut{0, ~0u, 0};
    u64 mass = r.mass;  // what top-k keeps
    if (r.k_bin >= 0 || q.by_list()) {
        if (r.k_bin >= 0) cut = descend(std::false_type(), r.k_left, [&](unsigned, int b) { return b == r.k_bin; });
        if (q.p < 1.0) {
            u64 s = 0;
            const bool by_token = cut.ties == ~0u, all = q.by_list();
            each([&](unsigned key, int b, unsigned token) {
                s += (all || b == r.k_bin) && (key > cut.key || (by_token && key == cut.key && token <= cut.token)) ? mass_at(key) : 0;
            });
            mass = r.k_mass + sum_all(s, sh.wave64) + (by_token ? 0 : (u64)cut.ties * mass_at(cut.key));
        }
    }
    if (q.p < 1.0) {
        const Cut k = cut;
        const u64 want = max((u64)ceil(q.p * (double)mass), (u64)1) - r.p_mass;
        cut = descend(std::true_type(), want, [&](unsigned key, int b) { return b >= r.p_lo && b <= r.p_hi && key >= k.key; });
        if (r.k_bin >= 0 && cut.key <= k.key)
            cut = cut.key == k.key ? Cut{k.key, min(cut.token, k.token), min(cut.ties, k.ties)} : k;
    }
    // what the chunks keep of their undecided tokens: those above the cut ...
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SAMPLE_SUBS; ++i) {
        sh.mass[i * TH + tid] = 0;
        sh.count[i * TH + tid] = 0;
    }
    __syncthreads();
    each([&](unsigned key, int, unsigned token) {
        if (key > cut.key) {
            const double v = weight(logit_of(key), t.top, q.c, sh.pow);
            if (v >= q.minp) atomicAdd(&sh.mass[token / SUB], mass_of(v));
        } else if (key == cut.key && token <= cut.token) {
            atomicAdd(&sh.count[token / SUB], 1u);
        }
    });
    __syncthreads();
    // ... and of the cut's key, the first tokens of the row
    unsigned ties[SAMPLE_SUBS], n = 0, all;
#pragma unroll
    for (int i = 0; i < SAMPLE_SUBS; ++i) n += ties[i] = sh.count[tid * SAMPLE_SUBS + i];
    const unsigned ties_before = scan_before(n, sh.wave32, all);
    const double v = weight(logit_of(cut.key), t.top, q.c, sh.pow);
    const u64 each_tie = v >= q.minp ? mass_of(v) : 0;
    n = ties_before;
#pragma unroll
    for (int i = 0; i < SAMPLE_SUBS; ++i) {
        kept[i] += sh.mass[tid * SAMPLE_SUBS + i] + min(ties[i], n < cut.ties ? cut.ties - n : 0u) * each_tie;
        n += ties[i];
    }
    pick<F32>(a, m, q, t, kept, &r, cut, ties, ties_before, sh);
}

template <bool F32>
void run(const SampleArgs &a, hipStream_t s) {
    const dim3 chunks((unsigned)((int64_t)a.M * a.chunks)), rows((unsigned)a.M);
    const bool borders = a.top_k || a.top_p;
    hipLaunchKernelGGL((sample_top_kernel<F32>), chunks, dim3(TH), 0, s, a);
    hipLaunchKernelGGL((sample_bins_kernel<F32>), chunks, dim3(TH), 0, s, a);
    if (!borders || !a.few) hipLaunchKernelGGL((sample_find_kernel<F32>), rows, dim3(TH), 0, s, a);
    if (!borders) return;
    if (a.few)
        hipLaunchKernelGGL((sample_list_kernel<F32, true>), chunks, dim3(TH), 0, s, a);
    else
        hipLaunchKernelGGL((sample_list_kernel<F32, false>), chunks, dim3(TH), 0, s, a);
    hipLaunchKernelGGL((sample_pick_kernel<F32>), rows, dim3(TH), 0, s, a);
}

}  // namespace

hipError_t launch_sample(const SampleArgs &a, bool x_f32, hipStream_t s) {
    x_f32 ? run<true>(a, s) : run<false>(a, s);
    return hipGetLastError();
}

}  // namespace qg
