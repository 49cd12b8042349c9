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
// Bound by memory: each [T][D] tensor crosses once (4096 x 3584 bf16 with a channel's gate: forward 27 to 29 us,
// backward 42 to 45, column sums 5 to 6: 4.1 to 4.3 TB/s; 16384 x 7168: 608 us, 5.0 TB/s).  A row is kept by one block because its
// length (up to 16384) fits the registers of at most 1024 threads.
#include "block_internal.h"
#include "common.h"

namespace moe {

namespace {

constexpr int kWaveRows = 8;  // rows of a block whose waves have a row each

// Sixteen bytes at an element's own alignment: where the width or a pointer is not a multiple of 16 bytes
// (TAIL), rows begin anywhere.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

template <bool TAIL>
__device__ __forceinline__ u32x4 ld16(const void *p)
{
    if constexpr (TAIL) return *(const u32x4_any *)p;
    return *(const u32x4 *)p;
}

template <bool TAIL>
__device__ __forceinline__ void st16(void *p, u32x4 v)
{
    if constexpr (TAIL)
        *(u32x4_any *)p = v;
    else
        *(u32x4 *)p = v;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// Eight elements as they lie in memory; with TAIL only the first n < 8 of a row's last group may exist.
template <int DT, bool TAIL>
struct Raw {
    static constexpr int kWords = DT == DT_F32 ? 8 : 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const void *p, size_t i, int n)
    {
        const char *q = (const char *)p + i * (DT == DT_F32 ? 4 : 2);
        if (!TAIL || n >= 8) {
#pragma unroll
            for (int k = 0; k < kWords / 4; k++) {
                const u32x4 v = ld16<TAIL>(q + 16 * k);
#pragma unroll
                for (int e = 0; e < 4; e++) w[4 * k + e] = v[e];
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < kWords; k++) w[k] = 0u;
#pragma unroll
        for (int e = 0; e < 7; e++) {
            if (e >= n) break;
            if constexpr (DT == DT_F32)
                w[e] = ((const uint32_t *)q)[e];
            else
                w[e >> 1] |= (uint32_t)((const uint16_t *)q)[e] << (16 * (e & 1));
        }
    }

    __device__ __forceinline__ float at(int e) const
    {
        if constexpr (DT == DT_F32) return __uint_as_float(w[e]);
        return __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
    }
};

template <bool TAIL>
__device__ __forceinline__ void ld_vec(const void *p, int dt, size_t i, int n, float (&f)[8])
{
    if (dt == DT_F32) {
        Raw<DT_F32, TAIL> r;
        r.load(p, i, n);
#pragma unroll
        for (int e = 0; e < 8; e++) f[e] = r.at(e);
    } else {
        Raw<DT_BF16, TAIL> r;
        r.load(p, i, n);
#pragma unroll
        for (int e = 0; e < 8; e++) f[e] = r.at(e);
    }
}

template <bool TAIL>
__device__ __forceinline__ void st_vec(void *p, int dt, size_t i, int n, const float (&f)[8])
{
    char *q = (char *)p + i * (dt == DT_F32 ? 4 : 2);
    if (!TAIL || n >= 8) {
        if (dt == DT_F32) {
            st16<TAIL>(q, __builtin_bit_cast(u32x4, f32x4{f[0], f[1], f[2], f[3]}));
            st16<TAIL>(q + 16, __builtin_bit_cast(u32x4, f32x4{f[4], f[5], f[6], f[7]}));
        } else {
            st16<TAIL>(q, u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])});
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; e++) {
        if (e >= n) break;
        if (dt == DT_F32)
            ((float *)q)[e] = f[e];
        else
            ((uint16_t *)q)[e] = (uint16_t)pack_bf16(f[e], 0.f);
    }
}

// The value that storing f as dt keeps.
__device__ __forceinline__ void round_to(int dt, float (&f)[8])
{
    if (dt == DT_F32) return;
#pragma unroll
    for (int e = 0; e < 8; e++) f[e] = (float)(__bf16)f[e];
}

// Sum over the threads of a row: a wave (WAVE), or the block of up to 16 waves.  scr: two rows of 16
// floats used in turn, so one barrier per sum is enough.
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float (*scr)[16], int &turn)
{
    const int wv = threadIdx.x >> 6, nw = (blockDim.x + 63) >> 6;
    v = wave_sum_f32(v);
    if (WAVE || nw == 1) return v;
    float *s = scr[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) s[wv] = v;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < nw; w++) t += s[w];
    return t;
}

// A row's thread has NV groups of eight columns, at 8 (tid + i team).  MAXT = 64: each wave of the block has
// a row of its own (up to 512 columns); else the block has it.
template <int MAXT, int NV, bool TAIL, int RT, int YT, int XT>
__global__ __launch_bounds__(MAXT == 64 ? 64 * kWaveRows : MAXT) void k_norm_fwd(NormArgs a)
{
    constexpr bool kWave = MAXT == 64;
    __shared__ float scr[2][16];
    const int team = kWave ? 64 : (int)blockDim.x, tid = kWave ? threadIdx.x & 63 : threadIdx.x, D = a.D;
    const int first = kWave ? (int)(blockIdx.x * kWaveRows + (threadIdx.x >> 6)) : (int)blockIdx.x;
    const float invD = 1.f / (float)D;
    int turn = 0;
    const int t = first;
    if (t >= a.T) return;
    const size_t row = (size_t)t * D;
    const bool full = a.gate == GATE_FULL && a.y;
    float z[NV][8], y[NV][8], g[NV][8];
    {
        Raw<RT, TAIL> nr[NV];
        Raw<YT, TAIL> ny[NV], ng[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = 8 * (tid + i * team);
            if (c >= D) continue;
            nr[i].load(a.r, row + c, D - c);
            if (a.y) ny[i].load(a.y, row + c, D - c);
            if (full) ng[i].load(a.g, row + c, D - c);
        }
        const float tg = a.gate == GATE_TOKEN && a.y ? a.beta * ((const float *)a.g)[t] : a.beta;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const bool in = 8 * (tid + i * team) < D;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                z[i][e] = in ? nr[i].at(e) : 0.f;
                y[i][e] = in && a.y ? ny[i].at(e) : 0.f;
                g[i][e] = in && full ? tg * ng[i].at(e) : tg;
            }
        }
    }
    if (a.y) {
        float ss = 0.f, ry = 1.f;
        if (a.post) {
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int e = 0; e < 8; e++) ss += y[i][e] * y[i][e];
            ss = row_sum<kWave>(ss, scr, turn);
            ry = 1.f / sqrtf(ss * invD + a.eps_post);
            if (a.rstd && tid == 0) a.rstd[t] = ry;
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = 8 * (tid + i * team);
            if (c >= D) continue;
            float w[8];
            if (a.post) {
                ld_vec<TAIL>(a.w_post, a.wt, c, D - c, w);
#pragma unroll
                for (int e = 0; e < 8; e++) y[i][e] = y[i][e] * ry * w[e];
            }
            if (a.gate == GATE_CHANNEL) {
                ld_vec<TAIL>(a.g, DT_F32, c, D - c, w);
#pragma unroll
                for (int e = 0; e < 8; e++) g[i][e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < 8; e++) z[i][e] = a.alpha * z[i][e] + g[i][e] * y[i][e];
            round_to(RT, z[i]);
            st_vec<TAIL>(a.r_out, RT, row + c, D - c, z[i]);
        }
    }
    if (!a.next) return;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < 8; e++) ss += z[i][e] * z[i][e];
    ss = row_sum<kWave>(ss, scr, turn);
    const float rz = 1.f / sqrtf(ss * invD + a.eps_next);
    if (a.rstd && tid == 0) a.rstd[a.T + t] = rz;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = 8 * (tid + i * team);
        if (c >= D) continue;
        float w[8];
        ld_vec<TAIL>(a.w_next, a.wt, c, D - c, w);
#pragma unroll
        for (int e = 0; e < 8; e++) w[e] = z[i][e] * rz * w[e];
        st_vec<TAIL>(a.x, XT, row + c, D - c, w);
    }
}

// FULL: the gate is MOE_GATE_FULL (its row held beside the others).
template <int MAXT, int NV, bool TAIL, bool FULL, int RT, int YT, int XT>
__global__ __launch_bounds__(MAXT == 64 ? 64 * kWaveRows : MAXT) void k_norm_bwd(NormArgs a)
{
    constexpr bool kWave = MAXT == 64;
    __shared__ float scr[2][16];
    const int team = kWave ? 64 : (int)blockDim.x, tid = kWave ? threadIdx.x & 63 : threadIdx.x, D = a.D;
    const int first = kWave ? (int)(blockIdx.x * kWaveRows + (threadIdx.x >> 6)) : (int)blockIdx.x;
    const float invD = 1.f / (float)D;
    int turn = 0;
    if (kWave && first >= a.T) return;  // a wave without a row has no partial row either
    float s1[NV][8], s2[NV][8], sg[NV][8];
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < 8; e++) s1[i][e] = s2[i][e] = sg[i][e] = 0.f;

    Raw<RT, TAIL> nd[NV], nz[NV];
    Raw<YT, TAIL> ny[NV], ng[FULL ? NV : 1];
    Raw<XT, TAIL> nx[NV];
    float nrz = 0.f, nry = 1.f, ngt = 1.f;
    const bool token = a.gate == GATE_TOKEN && a.y;
    auto fetch = [&](int t) {
        const size_t row = (size_t)t * D;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = 8 * (tid + i * team);
            if (c >= D) continue;
            if (a.next) {
                nx[i].load(a.dx, row + c, D - c);
                nz[i].load(a.r_out, row + c, D - c);
            }
            if (a.dr_out) nd[i].load(a.dr_out, row + c, D - c);
            if (a.y) ny[i].load(a.y, row + c, D - c);
            if constexpr (FULL) ng[i].load(a.g, row + c, D - c);
        }
        if (a.next) nrz = a.rstd[a.T + t];
        if (a.y && a.post) nry = a.rstd[t];
        if (token) ngt = ((const float *)a.g)[t];
    };
    // the next row is requested before the present one is worked on, where the registers hold both
    constexpr bool kAhead = NV == 1;
    const int stride = kWave ? (int)gridDim.x * kWaveRows : (int)gridDim.x;
    if (kAhead && first < a.T) fetch(first);
    for (int t = first; t < a.T; t += stride) {
        if (!kAhead) fetch(t);
        const size_t row = (size_t)t * D;
        float d[NV][8], y[NV][8], g[FULL ? NV : 1][8], dxw[NV][8], zn[NV][8];
        const float rz = nrz, ry = nry, gt = ngt;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const bool in = 8 * (tid + i * team) < D;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                d[i][e] = in && a.dr_out ? nd[i].at(e) : 0.f;
                y[i][e] = in && a.y ? ny[i].at(e) * ry : 0.f;  // y hat
                if constexpr (FULL) g[i][e] = in ? ng[i].at(e) : 0.f;
                dxw[i][e] = in && a.next ? nx[i].at(e) : 0.f;
                zn[i][e] = in && a.next ? nz[i].at(e) * rz : 0.f;
            }
        }
        if (kAhead && t + stride < a.T) fetch(t + stride);
        if (a.next) {
            float c2 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int c = 8 * (tid + i * team);
                if (c >= D) continue;
                float w[8];
                ld_vec<TAIL>(a.w_next, a.wt, c, D - c, w);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    s2[i][e] += dxw[i][e] * zn[i][e];
                    dxw[i][e] *= w[e];
                    c2 += dxw[i][e] * zn[i][e];
                }
            }
            c2 = row_sum<kWave>(c2, scr, turn) * invD;
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int e = 0; e < 8; e++) d[i][e] += rz * (dxw[i][e] - zn[i][e] * c2);
        }
        if (!a.y) {
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int c = 8 * (tid + i * team);
                if (c < D) st_vec<TAIL>(a.dr, RT, row + c, D - c, d[i]);
            }
            continue;
        }
        // S: sum over the row of beta (gate) d w1 yhat, the gate of a token left out
        float S = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = 8 * (tid + i * team);
            if (c >= D) continue;
            float w[8], o[8];
#pragma unroll
            for (int e = 0; e < 8; e++) o[e] = a.alpha * d[i][e];
            st_vec<TAIL>(a.dr, RT, row + c, D - c, o);
            float gc[8];
#pragma unroll
            for (int e = 0; e < 8; e++) w[e] = 1.f, gc[e] = 1.f;
            if constexpr (FULL) {
#pragma unroll
                for (int e = 0; e < 8; e++) gc[e] = g[i][e];
            } else {
                if (a.gate == GATE_CHANNEL) ld_vec<TAIL>(a.g, DT_F32, c, D - c, gc);
            }
            if (a.post) ld_vec<TAIL>(a.w_post, a.wt, c, D - c, w);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float bd = a.beta * d[i][e], q = bd * gc[e];  // q: dn without a token's gate
                o[e] = bd * y[i][e] * w[e];                           // beta d n
                s1[i][e] += q * gt * y[i][e];
                sg[i][e] += o[e];
                d[i][e] = q * w[e];
                S += d[i][e] * y[i][e];
            }
            if (a.gate == GATE_FULL && a.dg) st_vec<TAIL>(a.dg, YT, row + c, D - c, o);
        }
        if (a.post || (a.gate == GATE_TOKEN && a.dg)) S = row_sum<kWave>(S, scr, turn);
        if (a.gate == GATE_TOKEN && a.dg && tid == 0) ((float *)a.dg)[t] = S;
        const float cs = a.post ? S * invD : 0.f;
        const float f = gt * ry;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = 8 * (tid + i * team);
            if (c >= D) continue;
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; e++) o[e] = f * (d[i][e] - y[i][e] * cs);
            st_vec<TAIL>(a.dy, YT, row + c, D - c, o);
        }
    }
    float *p = a.part + (size_t)first * 3 * D;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = 8 * (tid + i * team);
        if (c >= D) continue;
        if (a.dw_post) st_vec<TAIL>(p, DT_F32, c, D - c, s1[i]);
        if (a.dw_next) st_vec<TAIL>(p + D, DT_F32, c, D - c, s2[i]);
        if (a.gate == GATE_CHANNEL && a.dg) st_vec<TAIL>(p + 2 * (size_t)D, DT_F32, c, D - c, sg[i]);
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
#pragma unroll 8
        for (int b = rg * per; b < min(nb, (rg + 1) * per); b++) v += a.part[((size_t)b * 3 + q) * a.D + c];
    s[rg][cx] = v;
    __syncthreads();
    if (rg == 0 && c < a.D) {
        v = 0.f;
        for (int k = 0; k < 32; k++) v += s[k][cx];
        if (q == 2 || a.wt == DT_F32)
            ((float *)out)[c] = v;
        else
            ((uint16_t *)out)[c] = (uint16_t)pack_bf16(v, 0.f);
    }
}

bool aligned16(const NormArgs &a)
{
    if (a.D % 8) return false;
    for (const void *p : {a.w_post, a.w_next, a.r, a.y, a.g, (const void *)a.r_out, (const void *)a.x, a.dr_out, a.dx, (const void *)a.dr,
                          (const void *)a.dy, (const void *)a.dg})
        if ((uintptr_t)p % 16) return false;
    return true;
}

template <int MAXT, int NV, bool TAIL, int RT, int YT, int XT>
void go(const NormArgs &a, bool bwd, int grid, hipStream_t s)
{
    const int groups = (a.D + 7) / 8, th = MAXT == 64 ? 64 * kWaveRows : 64 * ((groups + 64 * NV - 1) / (64 * NV));  // few idle lanes
    if (MAXT == 64) grid = (grid + kWaveRows - 1) / kWaveRows;
    if (bwd && a.gate == GATE_FULL && a.y)
        hipLaunchKernelGGL((k_norm_bwd<MAXT, NV, TAIL, true, RT, YT, XT>), dim3(grid), dim3(th), 0, s, a);
    else if (bwd)
        hipLaunchKernelGGL((k_norm_bwd<MAXT, NV, TAIL, false, RT, YT, XT>), dim3(grid), dim3(th), 0, s, a);
    else
        hipLaunchKernelGGL((k_norm_fwd<MAXT, NV, TAIL, RT, YT, XT>), dim3(grid), dim3(th), 0, s, a);
}

template <bool TAIL, int RT, int YT, int XT>
void go_width(const NormArgs &a, bool bwd, int grid, hipStream_t s)
{
    // a wave a row up to 512 columns (16384 rows of 128: 64 -> 37 us)
    if (a.D <= kWaveWidth)
        go<64, 1, TAIL, RT, YT, XT>(a, bwd, grid, s);
    else if (a.D <= 8192)
        go<1024, 1, TAIL, RT, YT, XT>(a, bwd, grid, s);
    else
        go<1024, 2, TAIL, RT, YT, XT>(a, bwd, grid, s);
}

template <int RT, int YT, int XT>
void go_types(const NormArgs &a, bool bwd, int grid, hipStream_t s)
{
    if (aligned16(a))
        go_width<false, RT, YT, XT>(a, bwd, grid, s);
    else
        go_width<true, RT, YT, XT>(a, bwd, grid, s);
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
    const int most = norm_parts(a.D), nb = a.T < most ? a.T : most;  // 0 rows: the column sums are zero
    if (nb > 0) dispatch(a, true, nb, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !(a.dw_post || a.dw_next || (a.gate == GATE_CHANNEL && a.dg))) return e;
    hipLaunchKernelGGL(k_norm_cols, dim3((unsigned)((a.D + 31) / 32), 3), dim3(1024), 0, s, a, nb);
    return hipGetLastError();
}

}  // namespace moe
