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
// is only raised when a score passes it by 8 (in powers of two: p <= 2^8, and
// 2^7 p is inside f16), so most steps neither exchange across lanes nor rescale
// O.  The value scales enter p as vs / vref with vref a power of two at least
// as large as every vs that the wave has met in its segment.  So 2^7 p vs / vref
// is what f16 rounds: to 2^-11 of it down to p vs / vref = 2^-21, below that
// by up to 2^-32.
//
// The work is a line of (request, head, group of 16 NR RS rows, step).  It is
// cut into one equal run for each of the workgroups that fit the GPU at once,
// so that requests of any lengths load it evenly; a run's part of one
// (request, head, row group) is a segment.  Where there are few of these
// (batch-one decode), a cut falls on each one's start too, so that no
// workgroup has two segments.  A workgroup's waves split the segment's steps
// (TS of them) and the rows (RS) and join in LDS; a second kernel joins the
// segments.  Short contexts are not cut (WHOLE_MAX_8, WHOLE_MAX_4).
//
// Bound by the cache's stream for up to 16 rows (131072 tokens, 4 heads of
// 256, E4M3: 46.5 us, 5.8 TB/s; 330693 tokens in 48 requests, 8 heads of 128,
// int8: 126 us, 5.4 TB/s; the joins 6.4 us each), by the vector unit's
// conversions, which each of the RS waves does for itself, and softmax for many
// (128 rows, 46784 tokens: 54.5 us, 340 TFLOP/s, join 10.2), by latency for
// short contexts (1021 tokens: 11.7 us) and windows (512 of 131072 tokens: 10.5).
#include "kv_attn_kernel.h"

namespace qg {

// Joins the segments of a (query token, head), where there are several: W
// waves for each (join_segments), one where rows are many, else eight.  Bound by
// latency: request, head of the workspace, segments in turn.
template <int D, int RW, int W>
__global__ void __launch_bounds__(512) kv_attn_join_kernel(KvAttnArgs) {
    constexpr int ROWS = 8 / W;
    __shared__ JoinLds<D, W> lds;
    Args &a = args();
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = wave % W;
    const int which = blockIdx.x * ROWS + wave / W;  // (request, token, head)
    const int r = which / (a.max_q * a.Hq), j = which / a.Hq % a.max_q, hq = which % a.Hq;
    if (r >= a.R) return;
    const Req rq = req_of<RW>(a, r);
    if (j >= rq.T) return;
    const int row = j * a.G + hq % a.G, pair = (hq / a.G) * rq.groups + row / RW;
    const int len = max(a.head[0], 1), before = a.head[1 + r];
    int w0, n;
    if (a.aligned) {
        n = (rq.units + len - 1) / len;
        w0 = before + pair * n;
    } else {
        const int x = before + pair * rq.units;
        w0 = x / len;
        n = (x + rq.units - 1) / len - w0 + 1;
    }
    if (n == 1) return;  // not cut: written already
    const int slot = w0 + (a.aligned ? 0 : r * a.Hkv * a.groups + pair);
    // (never so, unless another call wrote to the workspace in between)
    if (slot < 0 || n < 1 || n > a.part_slots || slot > a.part_slots - n) return;
    const size_t at = (size_t)slot * a.part_rows + row % RW, step = a.part_rows;
    join_segments<D, W>(a, lds, n, rq.q0 + j, hq, wi, lane, [&](int c) {
        return Part{a.part, a.part_ml, at + c * step};
    });
}

namespace {

constexpr int WAVES = 4;
// Contexts (max_len, or what a window leaves of it) up to here are not cut: a
// second launch would cost more than the steps that the waves of a workgroup
// then take in turn.  With 16 rows or fewer to a KV head, D <= 128, 8 waves
// take them.  Measured, 8 heads of 128, uncut against cut, one request and
// eight of them: 1024 tokens, 4 rows 11.8 us against 13.3 and 12.3 against
// 16.8, 1536 13.3 against 13.4 and 14.2 against 17.4.  Otherwise 4 waves: 512
// tokens, 32 rows 13.4 against 16.2 and 13.5 against 19.2, 64 rows 19.0
// against 17.2 and 18.9 against 22.7, 128 rows 27.6 against 19.8 and 28.4
// against 32.3; 768 tokens, 32 rows 15.1 against 16.5 and 15.2 against 22.1,
// 64 rows 23.4 against 18.2 and 23.7 against 27.0, 128 rows 37 against 23 and
// 38 against 33; D = 256 (4 heads), 512 tokens, 8 rows 12.4 against 15.5 and
// 12.6 against 16.6, 64 rows 29.9 against 18.0 and 30.6 against 24.3.
constexpr int WHOLE_WAVES = 8, WHOLE_MAX_8 = 1024, WHOLE_MAX_4 = 512;

template <bool E4M3, int D, int NR, int RS>
void run(const KvAttnArgs &a, hipStream_t s) {
    const unsigned grid = a.whole ? (unsigned)(a.R * a.Hkv * a.groups) : (unsigned)a.slots;
    if constexpr (RS == 1 && NR == 1 && D <= 128)
        if (a.whole) {
            hipLaunchKernelGGL((kv_attn_kernel<E4M3, D, NR, RS, WHOLE_WAVES>), dim3(grid), dim3(WHOLE_WAVES * 64), 0, s, a);
            return;
        }
    hipLaunchKernelGGL((kv_attn_kernel<E4M3, D, NR, RS, WAVES>), dim3(grid), dim3(WAVES * 64), 0, s, a);
    if (a.whole) return;
    const int64_t joins = (int64_t)a.R * a.max_q * a.Hq;
    if (joins >= 1024)
        hipLaunchKernelGGL((kv_attn_join_kernel<D, 16 * NR * RS, 1>), dim3((unsigned)((joins + 7) / 8)), dim3(512), 0, s, a);
    else
        hipLaunchKernelGGL((kv_attn_join_kernel<D, 16 * NR * RS, 8>), dim3((unsigned)joins), dim3(512), 0, s, a);
}

template <bool E4M3, int D>
void pick(const KvAttnArgs &a, hipStream_t s) {
    const Shape v = shape_of(D, a.max_q * a.G);
    if constexpr (D == 256)
        v.RS == 1 ? run<E4M3, D, 1, 1>(a, s) : v.RS == 2 ? run<E4M3, D, 1, 2>(a, s) : run<E4M3, D, 1, 4>(a, s);
    else if (v.NR == 1)
        run<E4M3, D, 1, 1>(a, s);
    else
        v.RS == 1 ? run<E4M3, D, 2, 1>(a, s) : v.RS == 2 ? run<E4M3, D, 2, 2>(a, s) : run<E4M3, D, 2, 4>(a, s);
}

}  // namespace

bool kv_attention_plan(int64_t R, int64_t Hkv, int64_t G, int64_t D, int64_t max_q, int64_t seen, KvAttnPlan *p) {
    const int64_t rows = max_q * G;
    const Shape v = shape_of((int)D, rows);
    const int64_t RW = 16 * v.NR * v.RS, groups = (rows + RW - 1) / RW, units = (seen + KV_STEP - 1) / KV_STEP + 1;
    p->groups = (int)groups;
    p->whole = seen <= (v.NR == 1 && v.RS == 1 && D <= 128 ? WHOLE_MAX_8 : WHOLE_MAX_4);
    // workgroups that run at once: 3 to a CU of the variants of up to 168
    // registers, else 2
    p->slots = 256 * (v.NR == 1 && D <= 128 ? 3 : 2);
    p->min_run = WAVES / v.RS;  // a step for each of the waves that split them
    p->part_rows = (int)(rows < RW ? rows : RW);
    // few (request, head, row group)s: a cut on each one's start.  Many: twice
    // as many runs as fit at once (330693 tokens in 48 requests of 8 heads:
    // 128 us, with one round of them 142, with four 128).  Few, with half or
    // three quarters of the runs: 0.9 to 1.2 times the time over 16 sizes;
    // with half as many again up to 1.4 times
    p->aligned = 4 * R * Hkv * groups <= p->slots;
    if (!p->aligned) p->slots *= 2;
    p->part_slots = p->whole ? 0 : p->slots + (p->aligned ? 0 : R * Hkv * groups);
    p->head_bytes = p->whole ? 0 : PART_HEAD;
    return R * Hkv * groups * units < (int64_t(1) << 31) - 65536;
}

hipError_t launch_kv_attention(const KvAttnArgs &a, int D, bool e4m3, hipStream_t s) {
    if (e4m3)
        D == 64 ? pick<true, 64>(a, s) : D == 128 ? pick<true, 128>(a, s) : pick<true, 256>(a, s);
    else
        D == 64 ? pick<false, 64>(a, s) : D == 128 ? pick<false, 128>(a, s) : pick<false, 256>(a, s);
    return hipGetLastError();
}

}  // namespace qg
