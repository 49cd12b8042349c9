// adamw.hip -- one AdamW step over many tensors (include/moe_block.h has the formulas).
//
// Bound by memory: a parameter's bytes cross once (twice for the gradient when the step is
// clipped): 198 M bf16 parameters with fp32 states and masters 1.06 ms (5.6 TB/s), 44 M fp32 parameters with
// 8-bit states 132 to 141 us (5.0 to 5.3 TB/s) and their gradients' norm 37 to 46.  The tensors' table lives in the caller's workspace and every tensor is cut into
// chunks; one launch covers all chunks of all tensors, a block per chunk, so that hundreds of
// small tensors cost one launch and large ones spread over the card.  A wave works on 256
// consecutive elements at a time, four to a lane, which is also the run that shares a scale of
// the 8-bit states, so a scale is one reduction over the wave's registers.
//
// Rounding: sums and products are kept as written (no contraction to fused operations), so the
// new moments do not depend on how the compiler pairs them and a state replays to the same bits.
#include <math.h>

#include "block_internal.h"
#include "common.h"

#pragma clang fp contract(off)

namespace moe {

namespace {

constexpr float kE4m3Max = 448.f, kFltMin = 1.17549435e-38f;

__device__ __forceinline__ int64_t chunk_elem0(const AdamTensor &t, int64_t c, int chunk_elems)
{
    return (c - (int64_t)t.chunk0) * chunk_elems;
}

// Four consecutive elements; those at or past the tensor's end (left of them valid) read as zero.
__device__ __forceinline__ void ld4(const void *p, int dt, bool vec, int64_t i, int64_t left, float (&f)[4])
{
    if (vec && left >= 4) {
        if (dt == DT_F32) {
            const f32x4 v = *(const f32x4 *)((const float *)p + i);
#pragma unroll
            for (int e = 0; e < 4; e++) f[e] = v[e];
        } else {
            const u32x2 v = *(const u32x2 *)((const uint16_t *)p + i);
#pragma unroll
            for (int e = 0; e < 2; e++) {
                f[2 * e] = __uint_as_float(v[e] << 16);
                f[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; e++)
        f[e] = e < left ? (dt == DT_F32 ? ((const float *)p)[i + e] : bf16_bits_to_f32(((const uint16_t *)p)[i + e])) : 0.f;
}

__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b)
{
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void st4(void *p, int dt, bool vec, int64_t i, int64_t left, const float (&f)[4])
{
    if (vec && left >= 4) {
        if (dt == DT_F32)
            *(f32x4 *)((float *)p + i) = f32x4{f[0], f[1], f[2], f[3]};
        else
            *(u32x2 *)((uint16_t *)p + i) = u32x2{bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3])};
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; e++)
        if (e < left) {
            if (dt == DT_F32)
                ((float *)p)[i + e] = f[e];
            else
                ((uint16_t *)p)[i + e] = (uint16_t)bf16x2_bits(f[e], 0.f);
        }
}

__device__ __forceinline__ uint32_t ld_codes(const void *p, bool vec, int64_t i, int64_t left)
{
    if (vec && left >= 4) return *(const uint32_t *)((const uint8_t *)p + i);
    uint32_t v = 0;
#pragma unroll
    for (int e = 0; e < 4; e++)
        if (e < left) v |= (uint32_t)((const uint8_t *)p)[i + e] << (8 * e);
    return v;
}

__device__ __forceinline__ void st_codes(void *p, bool vec, int64_t i, int64_t left, uint32_t v)
{
    if (vec && left >= 4) {
        *(uint32_t *)((uint8_t *)p + i) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; e++)
        if (e < left) ((uint8_t *)p)[i + e] = (uint8_t)(v >> (8 * e));
}

__device__ __forceinline__ void decode4(uint32_t c, float scale, float (&f)[4])
{
    f[0] = __builtin_amdgcn_cvt_f32_fp8((int)c, 0) * scale;
    f[1] = __builtin_amdgcn_cvt_f32_fp8((int)c, 1) * scale;
    f[2] = __builtin_amdgcn_cvt_f32_fp8((int)c, 2) * scale;
    f[3] = __builtin_amdgcn_cvt_f32_fp8((int)c, 3) * scale;
}

// Codes of four values of a run (their absolute maximum over the wave gives the scale).
__device__ __forceinline__ uint32_t encode4(const float (&f)[4], float &scale)
{
    const float top = wave_max_f32(fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
    scale = top * (1.f / kE4m3Max);
    if (scale < kFltMin) {
        scale = 0.f;
        return 0u;
    }
    // |f| / scale <= 448 (1 + 2^-22): rounds to at most the largest code, nothing to clamp.  One division a
    // run (with one an element the step was bound by its arithmetic: 44 M parameters 170 us, now 135); with
    // the correctly rounded reciprocal, the remainder's correction gives the correctly rounded quotient
    // (Markstein), so the codes are those of the division and a state's next step starts from the same bits.
    const float inv = 1.f / scale;
    float q[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float q0 = f[e] * inv;
        q[e] = __builtin_fmaf(__builtin_fmaf(-q0, scale, f[e]), inv, q0);
    }
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
}

// beta^t by squaring: one thread of one block waits for it, and pow() takes a microsecond.
__device__ double power(double beta, unsigned long long t)
{
    double r = 1.0;
    for (; t; t >>= 1, beta *= beta)
        if (t & 1) r *= beta;
    return r;
}

// Starts a step: counts it and puts its numbers where every block finds them.
__device__ void begin_step(const AdamArgs &a, float clip)
{
    const unsigned long long t = a.ctl->step + 1;
    const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
    a.ctl->step = t;
    a.ctl->clip = clip;
    a.ctl->lr = (float)lr;
    a.ctl->lr_m = (float)(lr / (1.0 - power(a.beta1, t)));
    a.ctl->root_v = (float)(1.0 / sqrt(1.0 - power(a.beta2, t)));
}

}  // namespace

__global__ void k_adam_put(AdamPut e, int n, AdamTensor *tab)
{
    const int w = sizeof(AdamTensor) / 4;
    const uint32_t *s = (const uint32_t *)e.t;
    for (int i = threadIdx.x; i < n * w; i += blockDim.x) ((uint32_t *)tab)[i] = s[i];
}

// tensor of each chunk: the last one whose first chunk is not behind it
__global__ __launch_bounds__(256) void k_adam_map(const AdamTensor *__restrict__ tab, int n, uint32_t *__restrict__ chunk_of, int64_t chunks)
{
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= chunks) return;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if ((int64_t)tab[mid].chunk0 <= c)
            lo = mid;
        else
            hi = mid;
    }
    chunk_of[c] = (uint32_t)lo;
}

__global__ void k_adam_set_step(AdamCtl *ctl, unsigned long long step)
{
    ctl->step = step;
}

// Sums of squares of the gradients, one fp64 number a block: fp32 within a lane's sixteen elements of a
// chunk, fp64 beyond.
__global__ __launch_bounds__(256) void k_adam_norm(AdamArgs a)
{
    __shared__ double s[4];
    const int tid = threadIdx.x;
    double sum = 0.0;
    for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        const AdamTensor &t = a.tab[a.chunk_of[c]];
        const int64_t e0 = chunk_elem0(t, c, a.chunk_elems), n = t.n;
        const void *const p = t.g;
        const int gt = t.gt;
        float q = 0.f;
        if (t.vec && gt == DT_F32 && e0 + a.chunk_elems <= n) {
            // a whole chunk: every load requested before the first is used
            const f32x4 *const v = (const f32x4 *)((const float *)p + e0) + tid;
            f32x4 g[4];
#pragma unroll
            for (int k = 0; k < 4; k++) g[k] = v[1024 * k < a.chunk_elems ? 256 * k : 0];
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (1024 * k < a.chunk_elems) q += (g[k][0] * g[k][0] + g[k][1] * g[k][1]) + (g[k][2] * g[k][2] + g[k][3] * g[k][3]);
        } else {
            for (int k = 4 * tid; k < a.chunk_elems && e0 + k < n; k += 1024) {
                float g[4];
                ld4(p, gt, t.vec, e0 + k, n - e0 - k, g);
                q += (g[0] * g[0] + g[1] * g[1]) + (g[2] * g[2] + g[3] * g[3]);
            }
        }
        sum += (double)q;
    }
    sum = wave_sum_f64(sum);
    if ((tid & 63) == 0) s[tid >> 6] = sum;
    __syncthreads();
    if (tid == 0) a.part[blockIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
}

// Begins the step; with clipping, from the nb blocks' sums added in order.  (A launch of its own: a last
// block found by a counter waits for hundreds of draws from it.)
__global__ __launch_bounds__(256) void k_adam_begin(AdamArgs a, int nb)
{
    __shared__ double s[4];
    const int tid = threadIdx.x;
    double sum = 0.0;
    for (int b = tid; b < nb; b += 256) sum += a.part[b];
    sum = wave_sum_f64(sum);
    if ((tid & 63) == 0) s[tid >> 6] = sum;
    __syncthreads();
    if (tid != 0) return;
    if (!a.clipped) return begin_step(a, 1.f);
    const double norm = sqrt((s[0] + s[1]) + (s[2] + s[3]));
    if (isfinite(norm))
        begin_step(a, (float)((double)a.max_norm / fmax(norm, (double)a.max_norm)));
    else
        a.ctl->clip = -1.f;  // the step is skipped
    if (a.norm_out) *a.norm_out = (float)norm;
}

// One chunk per block.
template <bool E4M3>
__global__ __launch_bounds__(256) void k_adam_step(AdamArgs a)
{
    const int tid = threadIdx.x, lane = tid & 63;
    const float clip = a.ctl->clip;
    if (clip < 0.f) return;  // a gradient norm that is not finite: nothing changes
    const int64_t c = blockIdx.x;
    const AdamTensor t = a.tab[a.chunk_of[c]];
    const float b1 = (float)a.beta1, b1c = (float)(1.0 - a.beta1), b2 = (float)a.beta2, b2c = (float)(1.0 - a.beta2);
    const float decay = (float)(1.0 - (double)a.ctl->lr * t.lr_scale * t.wd), lr = a.ctl->lr_m * t.lr_scale, iroot2 = a.ctl->root_v;
    const int64_t e0 = chunk_elem0(t, c, a.chunk_elems);
    void *const pp = t.master ? (void *)t.master : t.p;
    const int pt = t.master ? DT_F32 : t.pt;
    for (int k = 4 * tid; k < a.chunk_elems; k += 1024) {
        const int64_t i = e0 + k, left = t.n - i;
        if (i - 4 * lane >= t.n) break;  // the wave's whole run lies past the end
        float g[4], p[4], m[4], v[4], root[4];
        ld4(t.g, t.gt, t.vec, i, left, g);
        ld4(pp, pt, t.vec, i, left, p);
        const int64_t run = i / kQBlock;
        if constexpr (E4M3) {
            decode4(ld_codes(t.m, t.vec, i, left), t.ms[run], m);
            decode4(ld_codes(t.v, t.vec, i, left), t.vs[run], v);
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = v[e] * v[e];
        } else {
            ld4(t.m, DT_F32, t.vec, i, left, m);
            ld4(t.v, DT_F32, t.vec, i, left, v);
        }
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float gc = g[e] * clip;
            m[e] = m[e] * b1 + gc * b1c;
            v[e] = v[e] * b2 + gc * gc * b2c;
            root[e] = sqrtf(v[e]);
            // v_rcp_f32 is within 1 ulp: of the update, not of the parameter
            p[e] = p[e] * decay - lr * (m[e] * __builtin_amdgcn_rcpf(root[e] * iroot2 + a.eps));
        }
        st4(pp, pt, t.vec, i, left, p);
        if (t.master) st4(t.p, t.pt, t.vec, i, left, p);
        if constexpr (E4M3) {
            float sm, sv;
            const uint32_t cm = encode4(m, sm);
            uint32_t cv = encode4(root, sv);
            if (sv != 0.f)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (root[e] > 0.f && !(cv & (0xFFu << (8 * e)))) cv |= 1u << (8 * e);
            st_codes(t.m, t.vec, i, left, cm);
            st_codes(t.v, t.vec, i, left, cv);
            if (lane == 0) t.ms[run] = sm, t.vs[run] = sv;
        } else {
            st4(t.m, DT_F32, t.vec, i, left, m);
            st4(t.v, DT_F32, t.vec, i, left, v);
        }
    }
}

hipError_t launch_adam_put(const AdamTensor *host, int n, AdamTensor *tab, hipStream_t s)
{
    for (int i = 0; i < n; i += kAdamPut) {
        AdamPut e;
        const int m = n - i < kAdamPut ? n - i : kAdamPut;
        for (int j = 0; j < kAdamPut; j++) e.t[j] = host[i + (j < m ? j : 0)];
        hipLaunchKernelGGL(k_adam_put, dim3(1), dim3(256), 0, s, e, m, tab + i);
        const hipError_t r = hipGetLastError();
        if (r != hipSuccess) return r;
    }
    return hipSuccess;
}

hipError_t launch_adam_map(const AdamTensor *tab, int n, uint32_t *chunk_of, int64_t chunks, hipStream_t s)
{
    if (chunks == 0) return hipSuccess;
    hipLaunchKernelGGL(k_adam_map, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, s, tab, n, chunk_of, chunks);
    return hipGetLastError();
}

hipError_t launch_adam_set_step(AdamCtl *ctl, unsigned long long step, hipStream_t s)
{
    hipLaunchKernelGGL(k_adam_set_step, dim3(1), dim3(1), 0, s, ctl, step);
    return hipGetLastError();
}

hipError_t launch_adam_step(const AdamArgs &a, hipStream_t s)
{
    const int nb = !a.clipped ? 0 : a.chunks < kAdamNormBlocks ? (int)a.chunks : kAdamNormBlocks;
    if (nb > 0) hipLaunchKernelGGL(k_adam_norm, dim3((unsigned)nb), dim3(256), 0, s, a);
    hipLaunchKernelGGL(k_adam_begin, dim3(1), dim3(256), 0, s, a, nb);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.chunks == 0) return e;
    if (a.e4m3)
        hipLaunchKernelGGL((k_adam_step<true>), dim3((unsigned)a.chunks), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_adam_step<false>), dim3((unsigned)a.chunks), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
