// sv_head.cu -- output head with 4-bit weights and group scales (the formula
// stands at sv_head_w4 in include/sv.h).
#include <climits>
#include <cstdint>

#include "sv.h"
#include "sv_device.cuh"
#include "sv_host.h"

namespace sv {

struct HeadArgs {
    const uint8_t *codes;
    const void *scale;
    const uint8_t *zero;
    bool scale_f32, out_f32;
    int V, H, group, G;
    const __nv_bfloat16 *x;
    int B, P;
    const int32_t *lengths;
    int extra;
    void *out;
};

__device__ __forceinline__ bool scheduled(const HeadArgs &a, int t) {
    const int b = t / a.P, p = t - b * a.P;
    return !a.lengths || p < static_cast<long long>(__ldg(a.lengths + b)) + a.extra;
}

constexpr int kHeadTokens = 8;   // tokens per CTA

// One warp per vocabulary row, kHeadTokens tokens; a lane takes 16 bytes
// (32 codes, one group at most) at a time.
__global__ void __launch_bounds__(256) head_kernel(HeadArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int v = blockIdx.x * 8 + (threadIdx.x >> 5), t0 = blockIdx.y * kHeadTokens;
    if (v >= a.V) return;
    const int nt = min(kHeadTokens, a.B * a.P - t0);
    float acc[kHeadTokens] = {};
    for (int k = 32 * lane; k < a.H; k += 1024) {
        const int g = k / a.group;
        const long long sg = static_cast<long long>(v) * a.G + g;
        const float s = a.scale_f32 ? __ldg(static_cast<const float *>(a.scale) + sg)
                                    : ld_elem<2>(static_cast<const char *>(a.scale), sg);
        const float z = a.zero ? static_cast<float>(__ldg(a.zero + sg) & 15) : 8.f;
        const uint4 u = ld_stream(a.codes + static_cast<long long>(v) * (a.H / 2) + k / 2);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        for (int t = 0; t < nt; ++t) {
            const uint4 *x = reinterpret_cast<const uint4 *>(a.x + static_cast<long long>(t0 + t) * a.H + k);
            float part = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 xv = __ldg(x + q);
                const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    part = fmaf(bf16_lo(xw[e]), static_cast<float>(w[q] >> (8 * e) & 15u) - z, part);
                    part = fmaf(bf16_hi(xw[e]), static_cast<float>(w[q] >> (8 * e + 4) & 15u) - z, part);
                }
            }
            acc[t] = fmaf(s, part, acc[t]);
        }
    }
    for (int t = 0; t < nt; ++t) {
        float y = acc[t];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (lane == 0 && scheduled(a, t0 + t)) {
            const long long at = static_cast<long long>(t0 + t) * a.V + v;
            if (a.out_f32) static_cast<float *>(a.out)[at] = y;
            else static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(y);
        }
    }
}

static sv_status head_check(const sv_w4 *w, int B, int P) {
    if (!w) return SV_ERR_ARG;
    if (w->scale_dtype != SV_F32 && w->scale_dtype != SV_BF16) return SV_ERR_DTYPE;
    if (w->V < 1 || w->V > SV_MAX_V || w->H < 1 || w->H > SV_MAX_H ||
        (w->group != 32 && w->group != 64 && w->group != 128) || w->H % w->group)
        return SV_ERR_SHAPE;
    if (B < 0 || P < 1 || static_cast<long long>(B) * P > (1 << 20)) return SV_ERR_SHAPE;
    return SV_OK;
}

}  // namespace sv

extern "C" size_t sv_head_w4_workspace_bytes(const sv_w4 *weight, int B, int P) {
    if (sv::head_check(weight, B, P) != SV_OK) return 0;
    return 0;
}

extern "C" sv_status sv_head_w4(const sv_w4 *weight, const void *x, int B, int P,
                                const int32_t *lengths, int extra, void *out, sv_dtype out_dtype,
                                void *workspace, size_t workspace_bytes, void *stream) {
    sv::NvtxRange nvtx_range("sv_head_w4");
    if (const sv_status e = sv::head_check(weight, B, P)) return e;
    if (out_dtype != SV_F32 && out_dtype != SV_BF16) return SV_ERR_DTYPE;
    if (B == 0) return SV_OK;
    if (!weight->codes || !weight->scale || !x || !out) return SV_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(weight->codes) | reinterpret_cast<uintptr_t>(x)) & 15) return SV_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(weight->scale) & (weight->scale_dtype == SV_F32 ? 3 : 1)) return SV_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(out) & (out_dtype == SV_F32 ? 3 : 1)) return SV_ERR_ARG;
    const size_t need = sv_head_w4_workspace_bytes(weight, B, P);
    if (need > 0 && !workspace) return SV_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return SV_ERR_ARG;
    if (workspace_bytes < need) return SV_ERR_WORKSPACE;
    sv::HeadArgs a = {};
    a.codes = weight->codes; a.scale = weight->scale; a.zero = weight->zero;
    a.scale_f32 = weight->scale_dtype == SV_F32;
    a.out_f32 = out_dtype == SV_F32;
    a.V = weight->V; a.H = weight->H; a.group = weight->group; a.G = weight->H / weight->group;
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.B = B; a.P = P; a.lengths = lengths; a.extra = extra; a.out = out;
    const int M = B * P;
    const int ty = (M + sv::kHeadTokens - 1) / sv::kHeadTokens;
    if (ty > 65535) return SV_ERR_SHAPE;
    return sv::note_cuda(sv::launch_pdl(sv::head_kernel, dim3((a.V + 7) / 8, ty), dim3(256), 0,
                                        static_cast<cudaStream_t>(stream), a));
}
