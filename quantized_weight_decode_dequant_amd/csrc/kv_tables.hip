// Block tables and slot maps of the paged cache, from request lengths held on
// the GPU (a decode loop that never reads a length back).
//
// Request r keeps kept = min(keep, len) of its tokens and gets add new ones.
// It had H = ceil(len / page) pages and needs W = ceil((kept + add) / page):
// it gives back H - W pages or takes W - H.  With the requests in order and a
// request's pages in order, the released pages are numbered i = 0..Rel-1 and
// the wanted ones j = 0..A-1.  The free list is a stack S[0..n): wanted page
// j is released page j while there is one, then S[n-1-(j-Rel)]; a released
// page i >= A nobody took goes to S[n+Rel-1-i].  So a release undoes the
// extension before it, entry for entry.
//
// One workgroup does it all: three prefix sums over the requests (new tokens,
// released and wanted pages) in LDS, then one thread per page or token, which
// finds its request in the prefix sum by bisection.  Nothing is changed when
// the step cannot be done (status).
#include "kv_cache.h"

namespace qg {

namespace {

constexpr int TB = 1024;  // threads

struct Req {
    int kept, have, want;
};

__device__ __forceinline__ Req request(const KvTablesArgs &a, int r) {
    const int len = max(a.lens[r], 0);
    const int kept = a.keep ? min(max(a.keep[r], 0), len) : len;
    const long long len1 = (long long)kept + max(a.add[r], 0);
    Req q;
    q.kept = kept;
    q.have = (int)(((long long)len + a.page - 1) / a.page);
    q.want = (int)((len1 + a.page - 1) / a.page);
    return q;
}

// the last i with p[i] <= x, for p[0] = 0 <= x < p[n] ascending
__device__ __forceinline__ int find(const int *p, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

}  // namespace

__global__ void __launch_bounds__(TB) kv_tables_kernel(KvTablesArgs a) {
    extern __shared__ int lds[];
    const int R = a.R, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int *q0 = lds, *rel0 = lds + (R + 1), *get0 = lds + 2 * (R + 1);
    __shared__ long long wsum[3][TB / 64];
    __shared__ int wbad[TB / 64];

    // each thread sums a run of requests, then the runs are scanned
    const int per = (R + TB - 1) / TB;
    const int r0 = min(tid * per, R), r1 = min(r0 + per, R);
    long long s[3] = {0, 0, 0};
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        const Req q = request(a, r);
        s[0] += max(a.add[r], 0);
        s[1] += max(q.have - q.want, 0);
        s[2] += max(q.want - q.have, 0);
        bad |= q.want > a.max_blocks || q.have > a.max_blocks;
    }
    long long pre[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        long long v = s[k];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const long long u = __shfl_up(v, d);
            if (lane >= d) v += u;
        }
        pre[k] = v - s[k];
        if (lane == 63) wsum[k][wave] = v;
    }
    const bool wave_bad = __any(bad);
    if (lane == 0) wbad[wave] = wave_bad;
    __syncthreads();
    long long total[3] = {0, 0, 0};
    bool any_bad = false;
    for (int w = 0; w < TB / 64; ++w) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (w == wave) pre[k] += total[k];
            total[k] += wsum[k][w];
        }
        any_bad |= wbad[w] != 0;
    }
    const int n = *a.free_count;
    int status = 0;
    if (n < 0 || n > a.pages || total[2] > n + total[1] || n + total[1] - total[2] > a.pages) status |= 1;
    if (any_bad) status |= 2;
    if (total[0] > a.max_tokens) status |= 4;
    const bool ok = status == 0;
    // every thread has read the count before it is written
    __syncthreads();
    if (ok) {
        for (int r = r0; r < r1; ++r) {
            const Req q = request(a, r);
            q0[r] = (int)pre[0];
            rel0[r] = (int)pre[1];
            get0[r] = (int)pre[2];
            pre[0] += max(a.add[r], 0);
            pre[1] += max(q.have - q.want, 0);
            pre[2] += max(q.want - q.have, 0);
        }
        if (tid == 0) {
            q0[R] = (int)total[0];
            rel0[R] = (int)total[1];
            get0[R] = (int)total[2];
        }
    }
    __syncthreads();
    const int tokens = ok ? (int)total[0] : 0;
    for (int r = tid; r <= R; r += TB) a.q_start[r] = ok ? q0[r] : 0;
    if (tid == 0) *a.status = status;
    if (ok) {
        const int Rel = (int)total[1], A = (int)total[2];
        const auto released = [&](int i) {
            const int r = find(rel0, R, i);
            return (size_t)r * a.max_blocks + request(a, r).want + (i - rel0[r]);
        };
        // wanted pages: reads rows that shrink and the list, writes rows that grow
        for (int j = tid; j < A; j += TB) {
            const int r = find(get0, R, j);
            const int page = j < Rel ? a.table[released(j)] : a.free_pages[n - 1 - (j - Rel)];
            a.table[(size_t)r * a.max_blocks + request(a, r).have + (j - get0[r])] = page;
        }
        // left-over pages: to the list's end, which nothing above read
        for (int i = A + tid; i < Rel; i += TB) a.free_pages[n + Rel - 1 - i] = a.table[released(i)];
        __syncthreads();
        for (int i = tid; i < Rel; i += TB) a.table[released(i)] = -1;
        if (tid == 0) *a.free_count = n + Rel - A;
    }
    __syncthreads();
    for (int i = tid; i < a.max_tokens; i += TB) {
        int slot = -1, pos = 0;
        if (i < tokens) {
            const int r = find(q0, R, i);
            pos = request(a, r).kept + (i - q0[r]);
            slot = a.table[(size_t)r * a.max_blocks + pos / a.page] * a.page + pos % a.page;
        }
        a.slots[i] = slot;
        a.positions[i] = pos;
    }
    __syncthreads();
    if (ok)
        for (int r = tid; r < R; r += TB) a.lens[r] = request(a, r).kept + (q0[r + 1] - q0[r]);
}

hipError_t launch_kv_tables(const KvTablesArgs &a, hipStream_t s) {
    hipLaunchKernelGGL(kv_tables_kernel, dim3(1), dim3(TB), 3 * (a.R + 1) * sizeof(int), s, a);
    return hipGetLastError();
}

}  // namespace qg
