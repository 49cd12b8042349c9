// ffn_few.hip -- the gated feed-forward block's forward for few tokens (decode).
//
// With at most 64 tokens the weights' bytes are all there is to move: each is used for a few MFMAs at
// most.  A block owns a handful of output columns and the whole reduction, so that nothing has to be
// joined across blocks: 16 RT weight rows (of gate/up half of them gate, half up rows of the same
// columns, so h is formed in the block) times 16 NT tokens.  Its eight waves share the reduction in
// turns of 64 k, a whole 128-byte line of each row; weights go straight from memory into MFMA operands
// (lane l holds row l % 16, eight k from 8 (l / 16)), tokens likewise through the caches.  The waves'
// sums meet in LDS and are added in wave order.
// Bound by memory: at 3584 -> 6144 the gate and up rows are 88 MB, the down rows 44 MB; one token takes 17.7
// and 11.8 us (5.0 and 3.7 TB/s, a plain copy of such size 4.8).
#include <type_traits>

#include "block_internal.h"
#include "common.h"
#include "ffn_act.h"

namespace moe {

namespace {

constexpr int kFewWaves = 8;
constexpr int kTurn = 64;  // k of a wave's turn

struct FewArgs {
    int T, N, K;             // tokens, output columns, reduction
    const uint16_t *x;       // [PL][T][K]
    const uint16_t *w, *w2;  // [N][K]; gate/up: the gate and the up matrix
    int planes;              // gate/up: terms of h
    uint16_t *h;             // gate/up: unless null
    float *gu;               // gate/up: kept unless null
    void *y;                 // down
    int yt;
    bool acc;
};

__device__ __forceinline__ uint16_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// PL: planes of x whose sum is the operand.
template <int NT, int RT, int PL, bool GU, int ACT>
__global__ __launch_bounds__(64 * kFewWaves) void k_ffn_few(FewArgs a)
{
    constexpr int kCols = GU ? 8 * RT : 16 * RT;  // output columns of a block
    constexpr int U = RT + NT * PL <= 2 ? 4 : RT + NT * PL <= 4 ? 2 : 1;  // turns whose loads are requested together
    __shared__ f32x4 red[kFewWaves][RT * NT][64];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, li = lane & 15;
    const int n0 = blockIdx.x * kCols, K = a.K;

    // rows and tokens past the end repeat the last one; their results are not used
    const uint16_t *wp[RT], *xp[NT];
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const int r = 16 * i + li;  // gate/up: the first half of the block's rows gate, the second up
        const bool up = GU && r >= 8 * RT;
        const int col = min(n0 + (up ? r - 8 * RT : r), a.N - 1);
        wp[i] = (up ? a.w2 : a.w) + (size_t)col * K + 8 * g;
    }
#pragma unroll
    for (int j = 0; j < NT; j++) xp[j] = a.x + (size_t)min(16 * j + li, a.T - 1) * K + 8 * g;
    const size_t plane = (size_t)a.T * K;

    f32x4 acc[RT][NT];
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int j = 0; j < NT; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto turns = [&](auto N, int t) {
        constexpr int n = decltype(N)::value;
        bf16x8 w[n][RT][2], x[n][NT][PL][2];
#pragma unroll
        for (int u = 0; u < n; u++) {
            const int k = kTurn * (t + kFewWaves * u);
#pragma unroll
            for (int h = 0; h < 2; h++) {
#pragma unroll
                for (int i = 0; i < RT; i++) w[u][i][h] = as_bf16x8(*(const u32x4 *)(wp[i] + k + 32 * h));
#pragma unroll
                for (int j = 0; j < NT; j++)
#pragma unroll
                    for (int p = 0; p < PL; p++) x[u][j][p][h] = as_bf16x8(*(const u32x4 *)(xp[j] + p * plane + k + 32 * h));
            }
        }
#pragma unroll
        for (int u = 0; u < n; u++)
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int p = 0; p < PL; p++)
#pragma unroll
                    for (int i = 0; i < RT; i++)
#pragma unroll
                        for (int j = 0; j < NT; j++) acc[i][j] = mfma16(w[u][i][h], x[u][j][p][h], acc[i][j]);
    };
    const int whole = K / kTurn;
    int t = wv;
    for (; t + kFewWaves * (U - 1) < whole; t += kFewWaves * U) turns(std::integral_constant<int, U>(), t);
    for (; t < whole; t += kFewWaves) turns(std::integral_constant<int, 1>(), t);
    if (t == whole && K % kTurn) {
        // the reduction's end: K is a multiple of 8, so a lane's eight k are inside or outside together
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int k = kTurn * whole + 32 * h;
            const bool in = k + 8 * g < K;
            const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < RT; i++) {
                const bf16x8 w = as_bf16x8(in ? *(const u32x4 *)(wp[i] + k) : zero);
#pragma unroll
                for (int j = 0; j < NT; j++)
#pragma unroll
                    for (int p = 0; p < PL; p++)
                        acc[i][j] = mfma16(w, as_bf16x8(in ? *(const u32x4 *)(xp[j] + p * plane + k) : zero), acc[i][j]);
            }
        }
    }

    // lane l holds rows 4 (l / 16) + 0..3 of token l % 16; as floats: token 16, row
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int j = 0; j < NT; j++) red[wv][i * NT + j][4 * li + g] = acc[i][j];
    __syncthreads();
    auto sum = [&](int tile, int e) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWaves; w++) v += ((const float *)red[w][tile])[e];
        return v;
    };
    for (int e = tid; e < kCols * 16 * NT; e += 64 * kFewWaves) {
        const int c = e % kCols, tok = e / kCols, n = n0 + c;
        if (tok >= a.T || n >= a.N) continue;
        const int j = tok >> 4, tl = 16 * (tok & 15);
        if constexpr (GU) {
            const int ru = c + 8 * RT;  // the up row
            const float gv = sum((c >> 4) * NT + j, tl + (c & 15)), uv = sum((ru >> 4) * NT + j, tl + (ru & 15));
            if (a.gu) {
                a.gu[(size_t)tok * 2 * a.N + n] = gv;
                a.gu[(size_t)tok * 2 * a.N + a.N + n] = uv;
            }
            if (!a.h) continue;
            const float h = gated<ACT>(gv, uv), hi = (float)(__bf16)h;
            uint16_t *dst = a.h + (size_t)tok * a.N + n;
            *dst = bf16_bits(h);
            if (a.planes > 1) {  // the three terms whose sum is h
                const float m = fabsf(hi) < INFINITY ? h - hi : 0.f;
                dst[(size_t)a.T * a.N] = bf16_bits(m);
                dst[2 * (size_t)a.T * a.N] = bf16_bits(m - (float)(__bf16)m);
            }
        } else {
            float v = sum((c >> 4) * NT + j, tl + (c & 15));
            const size_t at = (size_t)tok * a.N + n;
            if (a.yt == DT_F32) {
                float *p = (float *)a.y + at;
                *p = a.acc ? *p + v : v;
            } else {
                uint16_t *p = (uint16_t *)a.y + at;
                if (a.acc) v += bf16_bits_to_f32(*p);
                *p = bf16_bits(v);
            }
        }
    }
}

template <int NT, int RT, int PL, bool GU, int ACT>
hipError_t go(const FewArgs &a, hipStream_t s)
{
    constexpr int cols = GU ? 8 * RT : 16 * RT;
    hipLaunchKernelGGL((k_ffn_few<NT, RT, PL, GU, ACT>), dim3((unsigned)((a.N + cols - 1) / cols)), dim3(64 * kFewWaves), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ffn_few_gate_up(const FfnArgs &a, uint16_t *h, int planes, float *gu, hipStream_t s)
{
    FewArgs f{};
    f.T = a.T, f.N = a.I, f.K = a.D, f.x = a.x, f.w = a.wg, f.w2 = a.wu, f.planes = planes, f.h = h, f.gu = gu;
    const bool situ = a.act == ACT_SITU;
    if (a.T <= 16) return situ ? go<1, 1, 1, true, ACT_SITU>(f, s) : go<1, 1, 1, true, ACT_SWIGLU>(f, s);
    if (a.T <= 32) return situ ? go<2, 2, 1, true, ACT_SITU>(f, s) : go<2, 2, 1, true, ACT_SWIGLU>(f, s);
    return situ ? go<4, 2, 1, true, ACT_SITU>(f, s) : go<4, 2, 1, true, ACT_SWIGLU>(f, s);
}

hipError_t launch_ffn_few_down(const FfnArgs &a, int planes, hipStream_t s)
{
    FewArgs f{};
    f.T = a.T, f.N = a.D, f.K = a.I, f.x = a.h, f.w = a.wd, f.y = a.y, f.yt = a.yt, f.acc = a.acc;
    if (a.T <= 16) return planes == 1 ? go<1, 1, 1, false, 0>(f, s) : go<1, 1, 3, false, 0>(f, s);
    if (a.T <= 32) return planes == 1 ? go<2, 1, 1, false, 0>(f, s) : go<2, 1, 3, false, 0>(f, s);
    return planes == 1 ? go<4, 1, 1, false, 0>(f, s) : go<4, 1, 3, false, 0>(f, s);
}

}  // namespace moe
