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
// Three kernels, a workgroup for each chunk of 4096 tokens of a row:
//   sample_top    the chunk's largest logit
//   sample_bins   counts and masses by bins; the row's last workgroup finds the
//                 borders' bins.  Rows without top-k and top-p end here.
//   sample_pick   the chunk's kept mass and list; the row's last workgroup
//                 finds the borders and the token
// "Last" is told by a counter that the first kernel clears: nobody waits.
#include "sample.h"

namespace qg {

namespace {

typedef unsigned long long u64;

constexpr int TH = SAMPLE_THREADS, E = SAMPLE_PER_THREAD, NB = SAMPLE_BINS;
constexpr float NEG_INF = -__builtin_inff();
constexpr double UNIT = 0x1p42;  // of masses

__device__ __forceinline__ float f32_of(unsigned w) { return __builtin_bit_cast(float, w); }
__device__ __forceinline__ unsigned bits_of(float f) { return __builtin_bit_cast(unsigned, f); }

// E logits from token `at` on; NaN past the row's end
template <bool F32>
__device__ __forceinline__ void load_logits(const void *logits, int64_t row, int at, int V, float (&x)[E]) {
    constexpr int N = F32 ? 4 : 8;  // logits of 16 bytes
    const char *p = (const char *)logits + (row + at) * (F32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < E; i += N) {
        if (at + i + N <= V) {
            u32x4_t w;
            __builtin_memcpy(&w, p + i * (F32 ? 4 : 2), 16);  // rows are aligned to an element only
#pragma unroll
            for (int e = 0; e < 4; ++e) {
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
};

__device__ __forceinline__ Ask ask_of(const SampleArgs &a, int m) {
    Ask q;
    const float T = a.temperature ? a.temperature[m] : 1.f;
    const int k = a.top_k ? a.top_k[m] : 0;
    const float p = a.top_p ? a.top_p[m] : 1.f, minp = a.min_p ? a.min_p[m] : 0.f;
    q.greedy = !(T > 0.f) || k == 1;
    q.c = 1.44269504088896340736 / (double)T;
    q.k = k > 0 && k < a.V ? k : 0;
    q.p = p < 1.f ? (double)p : 1.0;  // (NaN: off)
    q.minp = minp > 0.f ? fmin((double)minp, 1.0) : 0.0;
    return q;
}

// 2^-(j / 32), for weights
__device__ __forceinline__ void make_powers(double *pow) {
    if (threadIdx.x < 32) pow[threadIdx.x] = exp2(-(double)threadIdx.x * 0.03125);
}

// exp((x - top) / T): 2^-t by t = (32 n + j) / 32 + rest, |rest| <= 1/64, the
// rest's power by its series to the fifth order (2e-15).  0 of NaN.
__device__ __forceinline__ double weight(float x, float top, double c, const double *pow) {
    const double d = x == top ? 0.0 : (double)top - (double)x;
    const double t = fmin(d * c, 1100.0);
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

// 128 bins to an octave of the distance from the top, from 1/16 on.
__device__ __forceinline__ int bin_of(float x, float top) {
    const float d = x == top ? 0.f : top - x;
    return min(max((int)(bits_of(d) >> 16) - ((127 - 4) << 7), 0), NB - 1);
}

// Sum over the workgroup's threads before this one, and over all.
template <typename T>
__device__ __forceinline__ T scan_before(T v, T *waves, T &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    T upto = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const T u = __shfl_up(upto, d);
        if (lane >= d) upto += u;
    }
    __syncthreads();
    if (lane == 63) waves[wave] = upto;
    __syncthreads();
    T before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < TH / 64; ++w) {
        if (w < wave) before += waves[w];
        total += waves[w];
    }
    return before + upto - v;
}

__device__ __forceinline__ u64 sum_all(u64 v, u64 *waves) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    __syncthreads();
    if (lane == 0) waves[wave] = v;
    __syncthreads();
    u64 total = 0;
#pragma unroll
    for (int w = 0; w < TH / 64; ++w) total += waves[w];
    return total;
}

__device__ __forceinline__ float max_all(float v, float *waves) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    __syncthreads();
    if (lane == 0) waves[wave] = v;
    __syncthreads();
    v = waves[0];
#pragma unroll
    for (int w = 1; w < TH / 64; ++w) v = fmaxf(v, waves[w]);
    return v;
}

// What a workgroup keeps in LDS.
struct Shared {
    double pow[32];
    union {
        u64 wave64[TH / 64];
        unsigned wave32[TH / 64];
        float wavef[TH / 64];
    };
    u64 found64[2];
    unsigned found32[4];
    unsigned last;
    u64 mass[NB];     // by bin; later by digit
    unsigned count[NB];
    unsigned ties[TH];  // by chunk
};

// Whether this is the row's last workgroup in a kernel: what the others wrote
// before is then to be seen.
__device__ __forceinline__ bool arrive_last(unsigned *arrived, unsigned of, Shared &sh) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) sh.last = atomicAdd(arrived, 1u) == of - 1;
    __syncthreads();
    if (!sh.last) return false;
    __threadfence();
    return true;
}

// ------------------------------------------------------------------ the chunks' largest
template <bool F32>
__global__ void __launch_bounds__(TH) sample_top_kernel(SampleArgs a) {
    __shared__ float waves[TH / 64];
    __shared__ unsigned first;
    const int c = blockIdx.x % a.chunks, m = blockIdx.x / a.chunks, tid = threadIdx.x;
    float x[E];
    load_logits<F32>(a.logits, (int64_t)m * a.stride, c * SAMPLE_CHUNK + tid * E, a.V, x);
    if (a.top_k || a.top_p) {
        for (int i = c * TH + tid; i < NB; i += a.chunks * TH) {
            a.masses[(size_t)m * NB + i] = 0;
            a.counts[(size_t)m * NB + i] = 0;
        }
    }
    if (c == 0 && tid == 0) {
        a.rows[m].arrived[0] = a.rows[m].arrived[1] = 0;
        a.rows[m].done = 0;
    }
    float top = NEG_INF;
#pragma unroll
    for (int e = 0; e < E; ++e) top = fmaxf(top, x[e]);  // (past NaN)
    if (tid == 0) first = 0x7FFFFFFF;
    top = max_all(top, waves);
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int e = E - 1; e >= 0; --e)
        if (x[e] == top) at = c * SAMPLE_CHUNK + tid * E + e;
    if (at != 0x7FFFFFFF) atomicMin(&first, (unsigned)at);
    __syncthreads();
    if (tid == 0) {
        a.tops[(size_t)m * a.chunks + c] = top;
        a.top_at[(size_t)m * a.chunks + c] = (int)first;
    }
}

// ------------------------------------------------------------------ the token
// A row's cut in terms of its undecided tokens: those of larger keys are kept,
// and the first `ties` of this key.
struct Cut {
    unsigned key, ties;
};

// Whether a filter's border lies in this bin.
__device__ __forceinline__ bool undecided(const SampleRow &r, int b) {
    return (b >= r.p_lo && b <= r.p_hi) || b == r.k_bin;
}

// The token, from the chunks' kept masses (`mine`: of chunk tid) and, where
// there are filters, their numbers of the cut key's tokens (sh.ties).
template <bool F32>
__device__ void pick(const SampleArgs &a, int m, const Ask &q, float top, u64 mine, const SampleRow *row, Cut cut,
                     Shared &sh) {
    const int tid = threadIdx.x;
    u64 total;
    const u64 before = scan_before(mine, sh.wave64, total);
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
    if (mine > 0 && r >= before && r - before < mine) {
        sh.found32[0] = (unsigned)tid;
        sh.found64[0] = r - before;
    }
    __syncthreads();
    const int c = (int)sh.found32[0];
    r = sh.found64[0];
    unsigned ties_before = 0, n;
    if (row) {
        ties_before = scan_before(tid < c ? sh.ties[tid] : 0u, sh.wave32, n);
        ties_before = n;
    }
    float x[E];
    const int at = c * SAMPLE_CHUNK + tid * E;
    load_logits<F32>(a.logits, (int64_t)m * a.stride, at, a.V, x);
    // this thread's tokens of the cut key come after this many others
    unsigned mine_ties = 0;
    if (row) {
#pragma unroll
        for (int e = 0; e < E; ++e) mine_ties += x[e] == x[e] && key_of(x[e]) == cut.key && undecided(*row, bin_of(x[e], top));
        ties_before += scan_before(mine_ties, sh.wave32, n);
    }
    u64 w[E], sum = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const double v = weight(x[e], top, q.c, sh.pow);
        bool keep = v >= q.minp;
        if (row && x[e] == x[e]) {
            const int b = bin_of(x[e], top);
            const unsigned key = key_of(x[e]);
            if (undecided(*row, b)) {
                keep &= key > cut.key || (key == cut.key && ties_before < cut.ties);
                ties_before += key == cut.key;
            } else {
                keep &= b < row->full;
            }
        }
        w[e] = keep && x[e] == x[e] ? mass_of(v) : 0;
        sum += w[e];
    }
    u64 from = scan_before(sum, sh.wave64, sum);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (w[e] > 0 && r >= from && r - from < w[e]) {
            a.tokens[m] = at + e;
            if (a.logprobs)
                a.logprobs[m] = (float)log(weight(x[e], top, q.c, sh.pow) / ((double)total * (1.0 / UNIT)));
        }
        from += w[e];
    }
}

// ------------------------------------------------------------------ counts and masses by bins
template <bool F32>
__global__ void __launch_bounds__(TH) sample_bins_kernel(SampleArgs a) {
    __shared__ Shared sh;
    const int c = blockIdx.x % a.chunks, m = blockIdx.x / a.chunks, tid = threadIdx.x;
    SampleRow *row = a.rows + m;
    const Ask q = ask_of(a, m);
    float x[E];
    if (!q.greedy) load_logits<F32>(a.logits, (int64_t)m * a.stride, c * SAMPLE_CHUNK + tid * E, a.V, x);
    make_powers(sh.pow);
    const float mine = tid < a.chunks ? a.tops[(size_t)m * a.chunks + tid] : NEG_INF;
    const float top = max_all(mine, sh.wavef);
    if (q.greedy) {
        if (c != 0) return;
        if (tid == 0) sh.found32[0] = 0x7FFFFFFF;
        __syncthreads();
        if (tid < a.chunks && mine == top) atomicMin(&sh.found32[0], (unsigned)a.top_at[(size_t)m * a.chunks + tid]);
        __syncthreads();
        if (tid == 0) {
            const bool none = top == NEG_INF;
            a.tokens[m] = none ? -1 : (int)sh.found32[0];
            if (a.logprobs) a.logprobs[m] = none ? __builtin_nanf("") : 0.f;
            row->done = 1;
        }
        return;
    }
    const bool filters = q.filters() && top != NEG_INF;
    if (!filters) {
        u64 sum = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const double v = weight(x[e], top, q.c, sh.pow);
            sum += v >= q.minp && top != NEG_INF ? mass_of(v) : 0;  // (a row of -infinities has no token)
        }
        sum = sum_all(sum, sh.wave64);
        if (tid == 0) a.kept[(size_t)m * a.chunks + c] = sum;
    } else {
        for (int i = tid; i < NB; i += TH) {
            sh.mass[i] = 0;
            sh.count[i] = 0;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (x[e] == x[e]) {
                const int b = bin_of(x[e], top);
                if (q.k > 0) atomicAdd(&sh.count[b], 1u);
                if (q.p < 1.0) atomicAdd(&sh.mass[b], mass_of(weight(x[e], top, q.c, sh.pow)));
            }
        }
        __syncthreads();
        for (int i = tid; i < NB; i += TH) {
            if (sh.count[i]) atomicAdd(&a.counts[(size_t)m * NB + i], sh.count[i]);
            if (sh.mass[i]) atomicAdd(&a.masses[(size_t)m * NB + i], sh.mass[i]);
        }
    }
    if (!arrive_last(&row->arrived[0], (unsigned)a.chunks, sh)) return;
    if (!filters) {
        const u64 kept = tid < a.chunks ? a.kept[(size_t)m * a.chunks + tid] : 0;
        pick<F32>(a, m, q, top, kept, nullptr, Cut{0, 0}, sh);
        if (tid == 0) row->done = 1;
        return;
    }
    // the borders' bins: 8 consecutive bins a thread
    constexpr int PER = NB / TH;
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
        sh.found32[0] = NB;  // top-k's bin, the tokens before it
        sh.found64[0] = total;  // mass before it
        sh.found64[1] = total;  // and behind it
        sh.found32[2] = sh.found32[3] = NB;  // top-p's bins
    }
    __syncthreads();
    const bool by_k = q.k > 0 && (unsigned)q.k < tokens;  // (tokens: without NaN)
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
    const int k_bin = by_k ? (int)sh.found32[0] : -1;
    const unsigned k_left = sh.found32[1];
    __syncthreads();
    if (q.p < 1.0) {
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
    if (tid == 0) {
        const bool by_p = q.p < 1.0;
        const int p_lo = (int)sh.found32[2];
        row->p_lo = by_p ? p_lo : NB;
        row->p_hi = by_p ? min((int)sh.found32[3], NB - 1) : -1;
        row->p_mass = sh.found64[0];
        row->k_bin = k_bin;
        row->k_left = k_left;
        row->k_mass = lo;
        row->mass = total;
        row->full = by_p ? p_lo : by_k ? k_bin : NB;
        row->done = 0;
    }
}

// ------------------------------------------------------------------ the borders, and the token
// f(key) for each undecided token of the row, a wave a chunk, and end(chunk)
// behind each chunk's.
template <bool F32, typename Fn, typename End>
__device__ void each_undecided(const SampleArgs &a, int m, const SampleRow &r, float top, Fn f, End end) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int c = wave; c < a.chunks; c += TH / 64) {
        const size_t at = (size_t)m * a.chunks + c;
        const unsigned n = a.listed[at];
        if (n <= SAMPLE_LIST) {
            for (unsigned i = lane; i < n; i += 64) f(a.lists[at * SAMPLE_LIST + i]);
        } else {  // too many for the list: from the logits again
            const int stop = min((c + 1) * SAMPLE_CHUNK, a.V);
            for (int i = c * SAMPLE_CHUNK + lane; i < stop; i += 64) {
                const int64_t j = (int64_t)m * a.stride + i;
                const float x = F32 ? ((const float *)a.logits)[j] : f32_of((unsigned)((const uint16_t *)a.logits)[j] << 16);
                if (x == x && undecided(r, bin_of(x, top))) f(key_of(x));
            }
        }
        end(c);
    }
}

// Among the undecided tokens that `in` takes, the largest first: where `want`
// tokens are together (or, by mass, where the mass before and with them
// reaches `want`).  Digits of 8 bits from the top; `above` is what lies above
// the cut's key.
template <bool F32, bool MASS, typename In>
__device__ Cut descend(const SampleArgs &a, int m, const SampleRow &r, float top, double c, u64 want, u64 &above, In in,
                       Shared &sh) {
    unsigned prefix = 0;
    above = 0;
    unsigned here = 0;
    for (int shift = 24; shift >= (F32 ? 0 : 16); shift -= 8) {
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += TH) {
            sh.mass[i] = 0;
            sh.count[i] = 0;
        }
        __syncthreads();
        each_undecided<F32>(
            a, m, r, top,
            [&](unsigned key) {
                if (shift < 24 && (key >> (shift + 8)) != (prefix >> (shift + 8))) return;
                const float x = logit_of(key);
                if (!in(key, bin_of(x, top))) return;
                const unsigned d = 255u - ((key >> shift) & 255u);
                atomicAdd(&sh.count[d], 1u);
                if (MASS) atomicAdd(&sh.mass[d], mass_of(weight(x, top, c, sh.pow)));
            },
            [](int) {});
        __syncthreads();
        const unsigned n = sh.count[threadIdx.x];
        const u64 v = MASS ? sh.mass[threadIdx.x] : (u64)n;
        u64 total;
        const u64 before = above + scan_before(v, sh.wave64, total);
        if (threadIdx.x == 0) sh.found32[0] = 256;
        __syncthreads();
        if (before < want && before + v >= want) {
            sh.found32[0] = threadIdx.x;
            sh.found32[1] = n;
            sh.found64[0] = before;
        }
        __syncthreads();
        if (sh.found32[0] == 256) {  // (not reached: everything)
            above += total;
            return Cut{0, 0};
        }
        prefix |= (255u - sh.found32[0]) << shift;
        here = sh.found32[1];
        above = sh.found64[0];
    }
    if (!F32) prefix |= prefix & 0x80000000u ? 0u : 0xFFFFu;  // (the low half of a negative bf16's key)
    u64 ties = want - above;
    if (MASS) {
        const u64 w = mass_of(weight(logit_of(prefix), top, c, sh.pow));
        ties = w > 0 ? (ties + w - 1) / w : here;
    }
    return Cut{prefix, ties < here ? (unsigned)ties : here};
}

template <bool F32>
__global__ void __launch_bounds__(TH) sample_pick_kernel(SampleArgs a) {
    __shared__ Shared sh;
    const int c = blockIdx.x % a.chunks, m = blockIdx.x / a.chunks, tid = threadIdx.x;
    const SampleRow r = a.rows[m];
    if (r.done) return;
    const Ask q = ask_of(a, m);
    float x[E];
    load_logits<F32>(a.logits, (int64_t)m * a.stride, c * SAMPLE_CHUNK + tid * E, a.V, x);
    make_powers(sh.pow);
    const float top = max_all(tid < a.chunks ? a.tops[(size_t)m * a.chunks + tid] : NEG_INF, sh.wavef);
    u64 sum = 0;
    unsigned open = 0, n = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (!(x[e] == x[e])) continue;
        const int b = bin_of(x[e], top);
        if (b < r.full) {
            const double v = weight(x[e], top, q.c, sh.pow);
            sum += v >= q.minp ? mass_of(v) : 0;
        } else if (undecided(r, b)) {
            open |= 1u << e;
            ++n;
        }
    }
    sum = sum_all(sum, sh.wave64);
    unsigned all;
    unsigned place = scan_before(n, sh.wave32, all);
    const size_t at = (size_t)m * a.chunks + c;
    if (all <= SAMPLE_LIST) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (open >> e & 1) a.lists[at * SAMPLE_LIST + place++] = key_of(x[e]);
    }
    if (tid == 0) {
        a.kept[at] = sum;
        a.listed[at] = all;
    }
    if (!arrive_last(&a.rows[m].arrived[1], (unsigned)a.chunks, sh)) return;

    Cut cut{0, 0xFFFFFFFFu};
    u64 above, k_total = r.mass;
    unsigned k_key = 0;
    if (r.k_bin >= 0) {
        cut = descend<F32, false>(a, m, r, top, q.c, r.k_left, above, [&](unsigned, int b) { return b == r.k_bin; }, sh);
        k_key = cut.key;
        if (q.p < 1.0) {
            // top-k's mass: of the bins before, and of its bin's tokens that are kept
            u64 s = 0;
            each_undecided<F32>(
                a, m, r, top,
                [&](unsigned key) {
                    const float v = logit_of(key);
                    if (key > k_key && bin_of(v, top) == r.k_bin) s += mass_of(weight(v, top, q.c, sh.pow));
                },
                [](int) {});
            k_total = r.k_mass + sum_all(s, sh.wave64) + (u64)cut.ties * mass_of(weight(logit_of(k_key), top, q.c, sh.pow));
        }
    }
    if (q.p < 1.0) {
        const u64 want = max((u64)ceil(q.p * (double)k_total), (u64)1) - r.p_mass;
        const unsigned k_ties = cut.ties;
        cut = descend<F32, true>(a, m, r, top, q.c, want, above,
                                 [&](unsigned key, int b) { return b >= r.p_lo && b <= r.p_hi && key >= k_key; }, sh);
        if (r.k_bin >= 0 && cut.key <= k_key) cut = Cut{k_key, cut.key == k_key ? min(cut.ties, k_ties) : k_ties};
    }
    // what the chunks keep of their undecided tokens: those above the cut ...
    __syncthreads();
    const int lane = tid & 63;
    u64 more = 0;
    unsigned ties = 0;
    each_undecided<F32>(
        a, m, r, top,
        [&](unsigned key) {
            if (key > cut.key) {
                const double v = weight(logit_of(key), top, q.c, sh.pow);
                more += v >= q.minp ? mass_of(v) : 0;
            }
            ties += key == cut.key;
        },
        [&](int chunk) {
#pragma unroll
            for (int d = 32; d; d >>= 1) {
                more += __shfl_xor(more, d);
                ties += __shfl_xor(ties, d);
            }
            if (lane == 0) {
                sh.mass[chunk] = more;
                sh.ties[chunk] = ties;
            }
            more = 0;
            ties = 0;
        });
    __syncthreads();
    // ... and of the cut's key, the first tokens of the row
    u64 kept = 0;
    unsigned t;
    const unsigned mine = tid < a.chunks ? sh.ties[tid] : 0;
    const unsigned ties_before = scan_before(mine, sh.wave32, t);
    if (tid < a.chunks) {
        const unsigned take = min(mine, ties_before < cut.ties ? cut.ties - ties_before : 0u);
        const double v = take ? weight(logit_of(cut.key), top, q.c, sh.pow) : 0.0;
        kept = a.kept[(size_t)m * a.chunks + tid] + sh.mass[tid] + (take && v >= q.minp ? take * mass_of(v) : 0);
    }
    pick<F32>(a, m, q, top, kept, &r, cut, sh);
}

template <bool F32>
void run(const SampleArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.M * a.chunks));
    hipLaunchKernelGGL((sample_top_kernel<F32>), grid, dim3(TH), 0, s, a);
    hipLaunchKernelGGL((sample_bins_kernel<F32>), grid, dim3(TH), 0, s, a);
    if (a.top_k || a.top_p) hipLaunchKernelGGL((sample_pick_kernel<F32>), grid, dim3(TH), 0, s, a);
}

}  // namespace

hipError_t launch_sample(const SampleArgs &a, bool x_f32, hipStream_t s) {
    x_f32 ? run<true>(a, s) : run<false>(a, s);
    return hipGetLastError();
}

}  // namespace qg
