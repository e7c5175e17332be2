// New keys and values written into the paged 8-bit cache.
//
// Per page and head: s = max(s_old, amax * (1 / top)) with amax over the new
// tokens' finite values, 1 / top the fp32 nearest to 1/127 (int8) or 1/448
// (E4M3) and s_old = 0 where the first of the new tokens opens the page; inv = 1 / s; code = round(x *
// inv), clamped to +-top.  Where s grew, the page's codes are rounded again
// from code * (s_old / s).  Each of these steps is one correctly rounded
// fp32 operation (round to nearest even), so the codes do not depend on how
// the work is split.
//
// One workgroup per (run of slots that lie in one page, head, K or V).
#include "kv_cache.h"

namespace qg {

namespace {

constexpr int AP_T = 256;
constexpr float AP_TINY = 0x1p-100f;  // blocks below this are stored as zeros

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

template <bool E4M3>
__device__ __forceinline__ uint8_t encode(float z) {
    if (z != z) z = 0.f;
    if (E4M3) {
        z = fminf(fmaxf(z, -448.f), 448.f);
        return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(z, z, 0, false) & 0xFF);
    }
    return (uint8_t)(int8_t)(int)fminf(fmaxf(rintf(z), -127.f), 127.f);
}

template <bool E4M3>
__device__ __forceinline__ float decode(uint8_t c) {
    if (E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
    return (float)(int8_t)c;
}

__device__ __forceinline__ int place(bool value, int t, int d, int D) {
    if (value)
        return (t >> 5) * 32 * D + (d >> 5) * 1024 + ((t & 15) >> 2) * 256 + (d & 15) * 16 +
               ((d >> 4) & 1) * 8 + ((t >> 4) & 1) * 4 + (t & 3);
    return (t >> 4) * 16 * D + (d >> 4) * 256 + (t & 15) * 16 + (d & 15);
}

}  // namespace

template <bool E4M3>
__global__ void __launch_bounds__(AP_T) kv_append_kernel(KvAppendArgs a) {
    __shared__ int first_bad;
    __shared__ float wmax[AP_T / 64];
    const int tid = threadIdx.x;
    const int h = blockIdx.y;
    const bool value = blockIdx.z != 0;
    const uint16_t *X = value ? a.V : a.K;
    const int64_t stride = value ? a.v_stride : a.k_stride;
    const int D = a.D, page = a.page;
    constexpr float inv_top = E4M3 ? 1.f / 448.f : 1.f / 127.f;
    const int m1 = min((int)(blockIdx.x + 1) * a.chunk, a.M);
    for (int m = blockIdx.x * a.chunk; m < m1; ++m) {
        const int slot = a.slots[m];
        if (slot < 0 || slot >= a.slots_end) continue;
        const int off = slot % page;
        if (off != 0 && m > 0 && a.slots[m - 1] == slot - 1) continue;  // not the first of its run
        // length of the run
        __syncthreads();
        if (tid == 0) first_bad = min(page - off, a.M - m);
        __syncthreads();
        if (tid < page - off && m + tid < a.M && a.slots[m + tid] != slot + tid) atomicMin(&first_bad, tid);
        __syncthreads();
        const int n = first_bad;
        const uint16_t *x = X + (size_t)m * stride + (size_t)h * D;
        float amax = 0.f;
        for (int e = tid; e < n * D; e += AP_T) {
            const float f = fabsf(bf16_lo(x[(size_t)(e / D) * stride + e % D]));
            if (finite(f)) amax = fmaxf(amax, f);
        }
        for (int d = 32; d; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
        if ((tid & 63) == 0) wmax[tid >> 6] = amax;
        __syncthreads();
        for (int w = 0; w < AP_T / 64; ++w) amax = fmaxf(amax, wmax[w]);
        if (amax < AP_TINY) amax = 0.f;
        const size_t block = (size_t)(slot / page) * a.Hkv + h;
        uint8_t *codes = (value ? a.v : a.k) + block * page * D;
        float *scale = (value ? a.v_scales : a.k_scales) + block;
        const float s_old = off ? *scale : 0.f;
        const float s = fmaxf(s_old, amax * inv_top);
        const float inv = s > 0.f ? 1.f / s : 0.f;
        if (off && s > s_old) {
            const float ratio = s_old / s;
            for (int e = tid; e < page * D; e += AP_T) codes[e] = encode<E4M3>(decode<E4M3>(codes[e]) * ratio);
        }
        __syncthreads();
        for (int e = tid; e < n * D; e += AP_T) {
            const int t = e / D, d = e % D;
            codes[place(value, off + t, d, D)] = encode<E4M3>(bf16_lo(x[(size_t)t * stride + d]) * inv);
        }
        if (tid == 0) *scale = s;
    }
}

hipError_t launch_kv_append(const KvAppendArgs &args, bool e4m3, hipStream_t s) {
    KvAppendArgs a = args;
    a.chunk = a.M <= 1024 ? 1 : 16;
    const dim3 grid((unsigned)((a.M + a.chunk - 1) / a.chunk), (unsigned)a.Hkv, 2);
    if (e4m3)
        hipLaunchKernelGGL((kv_append_kernel<true>), grid, dim3(AP_T), 0, s, a);
    else
        hipLaunchKernelGGL((kv_append_kernel<false>), grid, dim3(AP_T), 0, s, a);
    return hipGetLastError();
}

}  // namespace qg
