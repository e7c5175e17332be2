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
// One workgroup does the requests and pages: three prefix sums over the
// requests (new tokens, released and wanted pages) in LDS, then one thread per
// page, which finds its request in the prefix sum by bisection, four of them
// in flight.  It also does the slots of up to SLOTS_HERE tokens; more are left
// to a second kernel over the whole GPU (1024 requests, 125k tokens: 82 us in
// one workgroup).  Latency bounds both: 4.4 us for one request, 10 to 11 and
// 7 for the two kernels at 1024 requests whose lengths grow by 125k tokens
// (3.9k pages) or fall back.  Nothing is changed when the step cannot be done
// (status).
#include "kv_cache.h"

namespace qg {

namespace {

constexpr int TB = 1024;           // threads
constexpr int SLOTS_HERE = 4096;   // tokens whose slots the first kernel writes
constexpr int FLIGHT = 4;          // pages of a thread whose loads are in flight together
constexpr int SLOTS_WG = 1024;     // tokens of a workgroup of the second one

struct Req {
    int kept, add, have, want;
};

__device__ __forceinline__ Req request(const KvTablesArgs &a, int r) {
    const int len = max(a.lens[r], 0);
    Req q;
    q.add = max(a.add[r], 0);
    q.kept = a.keep ? min(max(a.keep[r], 0), len) : len;
    q.have = (int)(((unsigned)len + a.page - 1) >> a.page_bits);
    q.want = (int)(((unsigned long long)q.kept + q.add + a.page - 1) >> a.page_bits);
    return q;
}

// Where token pos of request r lies; -1 on a page id outside the pool (which
// the shift could wrap into it).
__device__ __forceinline__ int slot_of(const KvTablesArgs &a, int r, int pos) {
    const int page = a.table[(size_t)r * a.max_blocks + (pos >> a.page_bits)];
    return page >= 0 && page < a.pages ? (page << a.page_bits) + (pos & (a.page - 1)) : -1;
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
    const int n = *a.free_count;
    long long s[3] = {0, 0, 0};
    Req first = {0, 0, 0, 0};  // the run's first request stays in registers
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        const Req q = request(a, r);
        if (r == r0) first = q;
        s[0] += q.add;
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
#pragma unroll
    for (int w = 0; w < TB / 64; ++w) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const long long v = wsum[k][w];
            if (w < wave) pre[k] += v;
            total[k] += v;
        }
        any_bad |= wbad[w] != 0;
    }
    int status = 0;
    if (n < 0 || n > a.pages || total[2] > n + total[1] || n + total[1] - total[2] > a.pages) status |= 1;
    if (any_bad) status |= 2;
    if (total[0] > a.max_tokens) status |= 4;
    const bool ok = status == 0;
    if (ok) {
        for (int r = r0; r < r1; ++r) {
            const Req q = r == r0 ? first : request(a, r);
            q0[r] = (int)pre[0];
            rel0[r] = (int)pre[1];
            get0[r] = (int)pre[2];
            a.q_start[r] = (int)pre[0];
            pre[0] += q.add;
            pre[1] += max(q.have - q.want, 0);
            pre[2] += max(q.want - q.have, 0);
        }
        if (tid == 0) {
            q0[R] = (int)total[0];
            rel0[R] = (int)total[1];
            get0[R] = (int)total[2];
            a.q_start[R] = (int)total[0];
        }
    } else {
        for (int r = tid; r <= R; r += TB) a.q_start[r] = 0;
    }
    if (tid == 0) *a.status = status;
    __syncthreads();
    const int tokens = ok ? (int)total[0] : 0;
    if (ok) {
        const int Rel = (int)total[1], A = (int)total[2];
        // where released page i lies in the table
        const auto released = [&](int i) {
            const int r = find(rel0, R, i);
            return (size_t)r * a.max_blocks + request(a, r).want + (i - rel0[r]);
        };
        // A released entry is read by the one thread whose page it becomes, or
        // that lists it, and cleared by it.  Wanted pages: from rows that
        // shrink and the list, to rows that grow.
        for (int j0 = tid; j0 < A; j0 += FLIGHT * TB) {
            size_t to[FLIGHT], from[FLIGHT];
            int page[FLIGHT];
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) {
                const int j = j0 + k * TB;
                if (j >= A) break;
                const int r = find(get0, R, j);
                to[k] = (size_t)r * a.max_blocks + request(a, r).have + (j - get0[r]);
                if (j < Rel) from[k] = released(j);
                page[k] = j < Rel ? a.table[from[k]] : a.free_pages[n - 1 - (j - Rel)];
            }
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) {
                const int j = j0 + k * TB;
                if (j >= A) break;
                a.table[to[k]] = page[k];
                if (j < Rel) a.table[from[k]] = -1;
            }
        }
        // left-over pages: to the list's end, which nothing above read
        for (int i0 = A + tid; i0 < Rel; i0 += FLIGHT * TB) {
            size_t from[FLIGHT];
            int page[FLIGHT];
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) {
                const int i = i0 + k * TB;
                if (i >= Rel) break;
                from[k] = released(i);
                page[k] = a.table[from[k]];
            }
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) {
                const int i = i0 + k * TB;
                if (i >= Rel) break;
                a.free_pages[n + Rel - 1 - i] = page[k];
                a.table[from[k]] = -1;
            }
        }
        if (tid == 0) *a.free_count = n + Rel - A;
    }
    if (a.max_tokens <= SLOTS_HERE) {
        __syncthreads();
        for (int i = tid; i < a.max_tokens; i += TB) {
            int slot = -1, pos = 0;
            if (i < tokens) {
                const int r = find(q0, R, i);
                pos = request(a, r).kept + (i - q0[r]);
                slot = slot_of(a, r, pos);
            }
            a.slots[i] = slot;
            a.positions[i] = pos;
        }
    }
    __syncthreads();
    if (ok)
        for (int r = r0; r < r1; ++r) {
            const Req q = r == r0 ? first : request(a, r);
            a.lens[r] = q.kept + q.add;
        }
}

// The slots of many tokens, from the lengths and tables as the first kernel
// left them.
__global__ void __launch_bounds__(256) kv_slots_kernel(KvTablesArgs a) {
    extern __shared__ int q0[];
    const int R = a.R, tid = threadIdx.x;
    for (int r = tid; r <= R; r += 256) q0[r] = a.q_start[r];
    __syncthreads();
    const int tokens = q0[R];
#pragma unroll
    for (int k = 0; k < SLOTS_WG / 256; ++k) {
        const int i = blockIdx.x * SLOTS_WG + k * 256 + tid;
        if (i >= a.max_tokens) break;
        int slot = -1, pos = 0;
        if (i < tokens) {
            const int r = find(q0, R, i);
            pos = a.lens[r] - (q0[r + 1] - i);
            slot = slot_of(a, r, pos);
        }
        a.slots[i] = slot;
        a.positions[i] = pos;
    }
}

hipError_t launch_kv_tables(const KvTablesArgs &args, hipStream_t s) {
    KvTablesArgs a = args;
    a.page_bits = __builtin_ctz(a.page);
    hipLaunchKernelGGL(kv_tables_kernel, dim3(1), dim3(TB), 3 * (a.R + 1) * sizeof(int), s, a);
    if (a.max_tokens > SLOTS_HERE)
        hipLaunchKernelGGL(kv_slots_kernel, dim3((a.max_tokens + SLOTS_WG - 1) / SLOTS_WG), dim3(256),
                           (a.R + 1) * sizeof(int), s, a);
    return hipGetLastError();
}

}  // namespace qg
