// Attention of requests that share a prefix: as kv_attention.hip, with the
// prefix's tokens read once for all rows of the call.
//
// A row's softmax runs over the prefix and over its request's own tokens; both
// leave (maximum, sum, values) segments, and a join makes them one.  Against
// the prefix all query tokens of all requests are rows of one product, so what
// is memory's work for one request becomes the matrix cores' for many.  Up to
// 16 rows to a KV head the prefix is one more entry on the requests' line of
// work, in one launch; above it is a line of its own, of groups of up to 256
// rows times equal parts of the prefix.
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
    if (rq.units <= 0) return s;
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

// Joins the segments of a (query token, head): W waves for each, D / 4 lanes 4
// dimensions each of one segment, as kv_attn_join_kernel does.
template <int D, int W>
__global__ void __launch_bounds__(512) kv_prefix_join_kernel(KvPrefixJoinArgs p) {
    constexpr int TD = D / 4, NG = W * 64 / TD, AHEAD = 8, ROWS = 8 / W;
    __shared__ f32x4_t so[W > 1 ? W : 1][TD];
    __shared__ float sl[W], smx[W];
    Args &a = *(Args *)__builtin_amdgcn_kernarg_segment_ptr();
    Args &b = *((Args *)__builtin_amdgcn_kernarg_segment_ptr() + 1);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = wave % W, tid = wi * 64 + lane, gi = tid / TD, d4 = tid % TD;
    const int which = blockIdx.x * ROWS + wave / W;  // (request, token, head)
    const int r = which / (a.max_q * a.Hq), j = which / a.Hq % a.max_q, hq = which % a.Hq;
    if (r >= a.R) return;
    const Req rq = req_of<16, KV_OWN>(a, r), pq = req_of<16, KV_PREFIX>(b, 0);
    if (j >= rq.T) return;
    const int head = hq / a.G, g = hq % a.G, prow = (rq.q0 - pq.q0 + j) * a.G + g;
    const Segments s = segments_of(p.own, rq, r, a.head[1 + r], max(a.head[0], 1), p.own_rw, head, j * a.G + g, a.aligned, a.Hkv * a.groups);
    Segments t = p.both ? segments_of(p.own, pq, a.R, a.head[1 + a.R], max(a.head[0], 1), p.own_rw, head, prow, a.aligned, a.Hkv * a.groups)
                        : pq.units > 0 ? segments_of(p.pre, pq, 0, 0, max(b.head[0], 1), p.pre_rw, head, prow, true, 0) : Segments{0, 0, 0};
    const float *part = p.both ? a.part : b.part, *part_ml = p.both ? a.part_ml : b.part_ml;
    const int n = s.n + t.n;
    float mx = NEG_INF;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
    for (int c0 = gi; c0 < n; c0 += NG * AHEAD) {
        f32x4_t v[AHEAD];
        f32x2_t ml[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int c = min(c0 + i * NG, n - 1);
            const bool own = c < s.n;
            const size_t at = own ? s.at + c * s.step : t.at + (c - s.n) * t.step;
            v[i] = *reinterpret_cast<const f32x4_t *>((own ? a.part : part) + at * D + 4 * d4);
            ml[i] = *reinterpret_cast<const f32x2_t *>((own ? a.part_ml : part_ml) + 2 * at);
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
        if (lane < TD) so[wi][lane] = o;
        if (lane == 0) {
            sl[wi] = l;
            smx[wi] = top;
        }
        __syncthreads();
        if (wi != 0) return;
        const float mine = top;
#pragma unroll
        for (int k = 1; k < W; ++k) top = fmaxf(top, smx[k]);
        const float own = top == NEG_INF ? 1.f : __builtin_amdgcn_exp2f(mine - top);
        o *= own;
        l *= own;
#pragma unroll
        for (int k = 1; k < W; ++k) {
            const float f = top == NEG_INF ? 1.f : __builtin_amdgcn_exp2f(smx[k] - top);
            o += so[k][lane % TD] * f;
            l = fmaf(sl[k], f, l);
        }
    }
    if (lane >= TD) return;
    const float f = l == 0.f ? 0.f : 1.f / l;
    const size_t to = (size_t)(rq.q0 + j) * a.out_stride + (size_t)hq * D + 4 * d4;
    o *= f;
    if (a.out_f32)
        *reinterpret_cast<f32x4_t *>((float *)a.out + to) = o;
    else
        *reinterpret_cast<u32x2_t *>((uint16_t *)a.out + to) = bf16x4(o);
}

// The prefix's variant for M * G rows to a KV head: as a request's up to 128
// rows; more go to 8 waves that share the converted codes.
struct PrefixShape {
    int NR, RS, waves;
    bool conv;
};

constexpr PrefixShape prefix_shape(int D, int64_t rows) {
    if (D == 64 && rows > 128) return {4, 4, 4, true};
    if (D == 128 && rows > 128) return {2, 8, 8, true};
    if (D == 256 && rows > 64) return {1, 8, 8, true};
    const Shape v = shape_of(D, rows);
    return {v.NR, v.RS, 4, false};
}

template <bool E4M3, int D, int NR, int RS, int WAVES, KvMode MODE, bool CONV>
void run_line(const KvAttnArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((kv_attn_kernel<E4M3, D, NR, RS, WAVES, MODE, CONV>), dim3((unsigned)a.slots), dim3(WAVES * 64), 0, s, a);
}

template <bool E4M3, int D, KvMode MODE>
void pick_line(const KvAttnArgs &a, int NR, int RS, hipStream_t s) {
    if (NR == 1 && RS == 1) run_line<E4M3, D, 1, 1, 4, MODE, false>(a, s);
    if constexpr (D == 256) {
        if (RS == 2) run_line<E4M3, D, 1, 2, 4, MODE, false>(a, s);
        if (RS == 4) run_line<E4M3, D, 1, 4, 4, MODE, false>(a, s);
        if constexpr (MODE == KV_PREFIX)
            if (RS == 8) run_line<E4M3, D, 1, 8, 8, MODE, true>(a, s);
    } else {
        if (NR == 2 && RS == 1) run_line<E4M3, D, 2, 1, 4, MODE, false>(a, s);
        if (RS == 2) run_line<E4M3, D, 2, 2, 4, MODE, false>(a, s);
        if (NR == 2 && RS == 4) run_line<E4M3, D, 2, 4, 4, MODE, false>(a, s);
        if constexpr (MODE == KV_PREFIX && D == 128)
            if (RS == 8) run_line<E4M3, D, 2, 8, 8, MODE, true>(a, s);
        if constexpr (MODE == KV_PREFIX && D == 64)
            if (NR == 4) run_line<E4M3, D, 4, 4, 4, MODE, true>(a, s);
    }
}

template <bool E4M3, int D>
void run(const KvAttnArgs &own, const KvAttnArgs &pre, const KvPrefixPlan &p, hipStream_t s) {
    const Shape v = shape_of(D, (int64_t)own.max_q * own.G);
    const PrefixShape w = prefix_shape(D, (int64_t)own.M * own.G);
    if (p.both) {
        run_line<E4M3, D, 1, 1, 4, KV_BOTH, false>(own, s);
    } else {
        pick_line<E4M3, D, KV_PREFIX>(pre, w.NR, w.RS, s);
        pick_line<E4M3, D, KV_OWN>(own, v.NR, v.RS, s);
    }
    KvPrefixJoinArgs j;
    j.own = own;
    j.pre = pre;
    j.own_rw = 16 * v.NR * v.RS;
    j.pre_rw = 16 * w.NR * w.RS;
    j.both = p.both;
    const int64_t joins = (int64_t)own.R * own.max_q * own.Hq;
    if (joins >= 1024)
        hipLaunchKernelGGL((kv_prefix_join_kernel<D, 1>), dim3((unsigned)((joins + 7) / 8)), dim3(512), 0, s, j);
    else
        hipLaunchKernelGGL((kv_prefix_join_kernel<D, 8>), dim3((unsigned)joins), dim3(512), 0, s, j);
}

}  // namespace

bool kv_prefix_plan(int64_t R, int64_t M, int64_t Hkv, int64_t G, int64_t D, int64_t max_q, int64_t max_len,
                    int64_t max_prefix, KvPrefixPlan *p) {
    const int64_t rows = max_q * G, all = M * G, steps = (max_prefix + KV_STEP - 1) / KV_STEP;
    const Shape v = shape_of((int)D, rows);
    const PrefixShape w = prefix_shape((int)D, all);
    const int64_t RW = 16 * v.NR * v.RS, PW = 16 * w.NR * w.RS;
    const int64_t groups = (rows + RW - 1) / RW, pgroups = (all + PW - 1) / PW, units = (max_len + KV_STEP - 1) / KV_STEP + 1;
    p->both = all <= 16 && rows <= 16;
    // the requests' line, cut as kv_attention_plan says
    KvAttnPlan &o = p->own;
    const int64_t starts = R * Hkv * groups + (p->both ? Hkv * pgroups : 0);
    int64_t most = R * Hkv * groups * units + (p->both ? Hkv * pgroups * (steps + 1) : 0);
    if (most >= (int64_t(1) << 31) - 65536) return false;
    o.groups = (int)groups;
    o.whole = false;
    o.slots = 256 * (v.NR == 1 && D <= 128 ? 3 : 2);
    o.min_run = 4 / v.RS;
    o.part_rows = (int)(p->both ? 16 : rows < RW ? rows : RW);
    o.aligned = 4 * starts <= o.slots;
    if (!o.aligned) o.slots *= 2;
    o.part_slots = o.slots + (o.aligned ? 0 : starts);
    o.head_bytes = PART_HEAD;
    p->own_starts = (int)starts;
    // the prefix's: parts of at least 8 steps, as many as fill the GPU best
    KvAttnPlan &q = p->pre;
    const int64_t pairs = Hkv * pgroups, fit = 256 * (w.conv ? 1 : w.NR == 1 && D <= 128 ? 3 : 2);
    if (pairs * (steps + 1) >= (int64_t(1) << 31) - 65536) return false;
    const int64_t longest = steps / 8 > 1 ? steps / 8 : 1, upto = longest < 4 * fit / pairs ? longest : 4 * fit / pairs;
    int64_t best = 1;
    double least = 1e30;
    for (int64_t k = 1; k <= upto; ++k) {
        // rounds of workgroups, each of its steps and of about 12 more of first loads and last sums
        const double cost = (double)((pairs * k + fit - 1) / fit) * ((double)((steps + k - 1) / k) + 12.0);
        if (cost < least) {
            least = cost;
            best = k;
        }
    }
    p->cuts = (int)best;
    q.groups = (int)pgroups;
    q.whole = false;
    q.slots = (int)(p->both ? 0 : pairs * best);
    q.min_run = w.conv ? 1 : 4 / w.RS;
    q.part_rows = (int)(all < PW ? all : PW);
    q.aligned = true;
    q.part_slots = q.slots;
    q.head_bytes = p->both ? 0 : PART_HEAD;
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
