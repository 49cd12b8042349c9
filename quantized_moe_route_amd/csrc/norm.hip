// norm.hip -- the RMS norms after a block and before the next one, fused with the block's gate
// and residual scale (include/moe_block.h has the formulas).
//
// Forward: one block holds one token's row in registers, so r, y and gate are read once and
// r_out and x written once; two block-wide sums (of y^2, then of the stored r_out^2).
// Backward, with z = r_out and the saved rz, ry (t a token, means over its row):
//   d    = dr_out + rz (dx w2 - z rz^2 mean(dx w2 z))
//   dn   = beta gate d,   dr = alpha d
//   dy   = ry (dn w1 - y ry^2 mean(dn w1 y))
//   dgate = beta d y ry w1,  dw1 = sum_t dn y ry,  dw2 = sum_t dx z rz
// A block walks rows t, t + gridDim, ... and keeps the column sums (dw1, dw2, dgate of
// MOE_GATE_CHANNEL) of its columns in fp32 registers; it writes them once as partial rows, which
// k_norm_cols adds in block order, so the sums have one fixed order.
// Bound by memory: each [T][D] tensor crosses once.  A row is kept by one block because its
// length (up to 16384) fits the registers of at most 1024 threads.
#include "block_internal.h"
#include "common.h"

namespace moe {

namespace {

template <int VEC>
__device__ __forceinline__ void ld_vec(const void *p, int dt, size_t i, float (&f)[VEC])
{
    if constexpr (VEC == 8) {
        if (dt == DT_F32) {
            const f32x4 a = *(const f32x4 *)((const float *)p + i), b = *(const f32x4 *)((const float *)p + i + 4);
#pragma unroll
            for (int e = 0; e < 4; e++) f[e] = a[e], f[4 + e] = b[e];
        } else {
            const u32x4 v = *(const u32x4 *)((const uint16_t *)p + i);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                f[2 * e] = __uint_as_float(v[e] << 16);
                f[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
            }
        }
    } else {
        f[0] = dt == DT_F32 ? ((const float *)p)[i] : bf16_bits_to_f32(((const uint16_t *)p)[i]);
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

template <int VEC>
__device__ __forceinline__ void st_vec(void *p, int dt, size_t i, const float (&f)[VEC])
{
    if constexpr (VEC == 8) {
        if (dt == DT_F32) {
            *(f32x4 *)((float *)p + i) = f32x4{f[0], f[1], f[2], f[3]};
            *(f32x4 *)((float *)p + i + 4) = f32x4{f[4], f[5], f[6], f[7]};
        } else {
            *(u32x4 *)((uint16_t *)p + i) = u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
        }
    } else {
        if (dt == DT_F32)
            ((float *)p)[i] = f[0];
        else
            ((uint16_t *)p)[i] = (uint16_t)pack_bf16(f[0], 0.f);
    }
}

// The value that storing f as dt keeps.
template <int VEC>
__device__ __forceinline__ void round_to(int dt, float (&f)[VEC])
{
    if (dt == DT_F32) return;
#pragma unroll
    for (int e = 0; e < VEC; e++) f[e] = (float)(__bf16)f[e];
}

// Sum over the block (up to 16 waves).  scr: two rows of 16 floats used in turn, so one barrier
// per sum is enough.
__device__ __forceinline__ float block_sum(float v, float (*scr)[16], int &turn)
{
    const int wv = threadIdx.x >> 6, nw = (blockDim.x + 63) >> 6;
    v = wave_sum_f32(v);
    if (nw == 1) return v;
    float *s = scr[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) s[wv] = v;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < nw; w++) t += s[w];
    return t;
}

// Elements of thread tid: NV groups of VEC at VEC (tid + i blockDim).
template <int VEC, int NV, int RT, int YT, int XT>
__global__ __launch_bounds__(1024) void k_norm_fwd(NormArgs a)
{
    __shared__ float scr[2][16];
    const int tid = threadIdx.x, D = a.D, t = blockIdx.x;
    const size_t row = (size_t)t * D;
    const float invD = 1.f / (float)D;
    int turn = 0;
    float z[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = VEC * (tid + i * (int)blockDim.x);
        if (c < D)
            ld_vec<VEC>(a.r, RT, row + c, z[i]);
        else
#pragma unroll
            for (int e = 0; e < VEC; e++) z[i][e] = 0.f;
    }
    if (a.y) {
        float y[NV][VEC], ss = 0.f, ry = 1.f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = VEC * (tid + i * (int)blockDim.x);
            if (c < D)
                ld_vec<VEC>(a.y, YT, row + c, y[i]);
            else
#pragma unroll
                for (int e = 0; e < VEC; e++) y[i][e] = 0.f;
        }
        if (a.post) {
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int e = 0; e < VEC; e++) ss += y[i][e] * y[i][e];
            ss = block_sum(ss, scr, turn);
            ry = 1.f / sqrtf(ss * invD + a.eps_post);
            if (a.rstd && tid == 0) a.rstd[t] = ry;
        }
        float tg = a.beta;
        if (a.gate == GATE_TOKEN) tg *= ((const float *)a.g)[t];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = VEC * (tid + i * (int)blockDim.x);
            if (c >= D) continue;
            float w[VEC], g[VEC];
            if (a.post) {
                ld_vec<VEC>(a.w_post, a.wt, c, w);
#pragma unroll
                for (int e = 0; e < VEC; e++) y[i][e] = y[i][e] * ry * w[e];
            }
            if (a.gate == GATE_CHANNEL) ld_vec<VEC>(a.g, DT_F32, c, g);
            if (a.gate == GATE_FULL) ld_vec<VEC>(a.g, YT, row + c, g);
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                const float s = a.gate == GATE_CHANNEL || a.gate == GATE_FULL ? tg * g[e] : tg;
                z[i][e] = a.alpha * z[i][e] + s * y[i][e];
            }
            round_to<VEC>(RT, z[i]);
            st_vec<VEC>(a.r_out, RT, row + c, z[i]);
        }
    }
    if (!a.next) return;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < VEC; e++) ss += z[i][e] * z[i][e];
    ss = block_sum(ss, scr, turn);
    const float rz = 1.f / sqrtf(ss * invD + a.eps_next);
    if (a.rstd && tid == 0) a.rstd[a.T + t] = rz;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = VEC * (tid + i * (int)blockDim.x);
        if (c >= D) continue;
        float w[VEC];
        ld_vec<VEC>(a.w_next, a.wt, c, w);
#pragma unroll
        for (int e = 0; e < VEC; e++) w[e] = z[i][e] * rz * w[e];
        st_vec<VEC>(a.x, XT, row + c, w);
    }
}

template <int VEC, int NV, int RT, int YT, int XT>
__global__ __launch_bounds__(1024) void k_norm_bwd(NormArgs a)
{
    __shared__ float scr[2][16];
    const int tid = threadIdx.x, D = a.D;
    const float invD = 1.f / (float)D;
    int turn = 0;
    float s1[NV][VEC], s2[NV][VEC], sg[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < VEC; e++) s1[i][e] = s2[i][e] = sg[i][e] = 0.f;

    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t row = (size_t)t * D;
        float d[NV][VEC], y[NV][VEC], dxw[NV][VEC];
        const float rz = a.next ? a.rstd[a.T + t] : 0.f;
        const float ry = a.y && a.post ? a.rstd[t] : 1.f;
        float c2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = VEC * (tid + i * (int)blockDim.x);
            const bool in = c < D;
#pragma unroll
            for (int e = 0; e < VEC; e++) d[i][e] = y[i][e] = dxw[i][e] = 0.f;
            if (!in) continue;
            if (a.dr_out) ld_vec<VEC>(a.dr_out, RT, row + c, d[i]);
            if (a.y) ld_vec<VEC>(a.y, YT, row + c, y[i]);
            if (a.next) {
                float z[VEC], w[VEC];
                ld_vec<VEC>(a.dx, XT, row + c, dxw[i]);
                ld_vec<VEC>(a.r_out, RT, row + c, z);
                ld_vec<VEC>(a.w_next, a.wt, c, w);
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    const float zn = z[e] * rz;
                    s2[i][e] += dxw[i][e] * zn;
                    dxw[i][e] *= w[e];
                    c2 += dxw[i][e] * zn;
                }
            }
        }
        if (a.next) {
            c2 = block_sum(c2, scr, turn) * invD;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int c = VEC * (tid + i * (int)blockDim.x);
                if (c >= D) continue;
                float z[VEC];
                ld_vec<VEC>(a.r_out, RT, row + c, z);
#pragma unroll
                for (int e = 0; e < VEC; e++) d[i][e] += rz * (dxw[i][e] - z[e] * rz * c2);
            }
        }
        if (!a.y) {
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int c = VEC * (tid + i * (int)blockDim.x);
                if (c < D) st_vec<VEC>(a.dr, RT, row + c, d[i]);
            }
            continue;
        }
        const float gt = a.gate == GATE_TOKEN ? ((const float *)a.g)[t] : 1.f;
        // S = mean over the row of (gate) d w1 yhat, the gate of a token left out
        float S = 0.f;
        float dn[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = VEC * (tid + i * (int)blockDim.x);
#pragma unroll
            for (int e = 0; e < VEC; e++) dn[i][e] = 0.f;
            if (c >= D) continue;
            float w[VEC], g[VEC], o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; e++) w[e] = 1.f, g[e] = 1.f;
            if (a.post) ld_vec<VEC>(a.w_post, a.wt, c, w);
            if (a.gate == GATE_CHANNEL) ld_vec<VEC>(a.g, DT_F32, c, g);
            if (a.gate == GATE_FULL) ld_vec<VEC>(a.g, YT, row + c, g);
#pragma unroll
            for (int e = 0; e < VEC; e++) o[e] = a.alpha * d[i][e];
            st_vec<VEC>(a.dr, RT, row + c, o);
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                const float yh = y[i][e] * ry, bd = a.beta * d[i][e];
                o[e] = bd * yh * w[e];                       // beta d n
                const float q = bd * g[e];                   // dn without a token's gate
                s1[i][e] += q * gt * yh;
                sg[i][e] += o[e];
                dn[i][e] = q * w[e];
                S += dn[i][e] * yh;
                y[i][e] = yh;
            }
            if (a.gate == GATE_FULL && a.dg) st_vec<VEC>(a.dg, YT, row + c, o);
        }
        if (a.post || (a.gate == GATE_TOKEN && a.dg)) S = block_sum(S, scr, turn);
        if (a.gate == GATE_TOKEN && a.dg && tid == 0) ((float *)a.dg)[t] = S;
        const float cs = a.post ? S * invD : 0.f;
        const float f = gt * ry;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = VEC * (tid + i * (int)blockDim.x);
            if (c >= D) continue;
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; e++) o[e] = f * (dn[i][e] - y[i][e] * cs);
            st_vec<VEC>(a.dy, YT, row + c, o);
        }
    }
    float *p = a.part + (size_t)blockIdx.x * 3 * D;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = VEC * (tid + i * (int)blockDim.x);
        if (c >= D) continue;
        if (a.dw_post) st_vec<VEC>(p, DT_F32, c, s1[i]);
        if (a.dw_next) st_vec<VEC>(p + D, DT_F32, c, s2[i]);
        if (a.gate == GATE_CHANNEL && a.dg) st_vec<VEC>(p + 2 * (size_t)D, DT_F32, c, sg[i]);
    }
}

// Column sums of the nb partial rows of one output (blockIdx.y: 0 dw_post, 1 dw_next, 2 dgate):
// 32 columns a block, 32 groups of rows, each in order, then the groups in order.
__global__ __launch_bounds__(1024) void k_norm_cols(NormArgs a, int nb)
{
    __shared__ float s[32][33];
    const int q = blockIdx.y, cx = threadIdx.x & 31, rg = threadIdx.x >> 5, c = blockIdx.x * 32 + cx;
    void *out = q == 0 ? a.dw_post : q == 1 ? a.dw_next : a.gate == GATE_CHANNEL ? a.dg : nullptr;
    if (!out) return;
    const int per = (nb + 31) / 32;
    float v = 0.f;
    if (c < a.D)
        for (int b = rg * per; b < min(nb, (rg + 1) * per); b++) v += a.part[((size_t)b * 3 + q) * a.D + c];
    s[rg][cx] = v;
    __syncthreads();
    if (rg == 0 && c < a.D) {
        v = 0.f;
        for (int k = 0; k < 32; k++) v += s[k][cx];
        const float o[1] = {v};
        st_vec<1>(out, q == 2 ? DT_F32 : a.wt, c, o);
    }
}

bool wide(const NormArgs &a)
{
    if (a.D % 8) return false;
    for (const void *p : {a.w_post, a.w_next, a.r, a.y, a.g, (const void *)a.r_out, (const void *)a.x, a.dr_out, a.dx, (const void *)a.dr,
                          (const void *)a.dy, (const void *)a.dg})
        if ((uintptr_t)p % 16) return false;
    return true;
}

// Threads so that NV groups of VEC cover the row with few idle lanes.
int threads_for(int D, int vec, int nv)
{
    const int groups = (D + vec - 1) / vec;
    return 64 * ((groups + 64 * nv - 1) / (64 * nv));
}

template <int VEC, int NV, int RT, int YT, int XT>
void go(const NormArgs &a, bool bwd, int grid, hipStream_t s)
{
    const int th = threads_for(a.D, VEC, NV);
    if (bwd)
        hipLaunchKernelGGL((k_norm_bwd<VEC, NV, RT, YT, XT>), dim3(grid), dim3(th), 0, s, a);
    else
        hipLaunchKernelGGL((k_norm_fwd<VEC, NV, RT, YT, XT>), dim3(grid), dim3(th), 0, s, a);
}

template <int RT, int YT, int XT>
void go_types(const NormArgs &a, bool bwd, int grid, hipStream_t s)
{
    if (!wide(a))
        go<1, 16, RT, YT, XT>(a, bwd, grid, s);
    else if (a.D <= 8192)
        go<8, 1, RT, YT, XT>(a, bwd, grid, s);
    else
        go<8, 2, RT, YT, XT>(a, bwd, grid, s);
}

void dispatch(const NormArgs &a, bool bwd, int grid, hipStream_t s)
{
    switch ((a.rt == DT_BF16) * 4 + (a.yt == DT_BF16) * 2 + (a.xt == DT_BF16)) {
    case 0: go_types<DT_F32, DT_F32, DT_F32>(a, bwd, grid, s); break;
    case 1: go_types<DT_F32, DT_F32, DT_BF16>(a, bwd, grid, s); break;
    case 2: go_types<DT_F32, DT_BF16, DT_F32>(a, bwd, grid, s); break;
    case 3: go_types<DT_F32, DT_BF16, DT_BF16>(a, bwd, grid, s); break;
    case 4: go_types<DT_BF16, DT_F32, DT_F32>(a, bwd, grid, s); break;
    case 5: go_types<DT_BF16, DT_F32, DT_BF16>(a, bwd, grid, s); break;
    case 6: go_types<DT_BF16, DT_BF16, DT_F32>(a, bwd, grid, s); break;
    default: go_types<DT_BF16, DT_BF16, DT_BF16>(a, bwd, grid, s); break;
    }
}

}  // namespace

hipError_t launch_norm_forward(const NormArgs &a, hipStream_t s)
{
    dispatch(a, false, a.T, s);
    return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs &a, hipStream_t s)
{
    const int nb = a.T < kNormBlocks ? a.T : kNormBlocks;  // 0 rows: the column sums are zero
    if (nb > 0) dispatch(a, true, nb, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !(a.dw_post || a.dw_next || (a.gate == GATE_CHANNEL && a.dg))) return e;
    hipLaunchKernelGGL(k_norm_cols, dim3((unsigned)((a.D + 31) / 32), 3), dim3(1024), 0, s, a, nb);
    return hipGetLastError();
}

}  // namespace moe
