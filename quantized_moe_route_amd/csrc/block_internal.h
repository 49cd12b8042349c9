// block_internal.h -- arguments and launchers of the dense block operators (include/moe_block.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// ---- norms around a block (norm.hip)
enum { GATE_NONE = 0, GATE_CHANNEL = 1, GATE_TOKEN = 2, GATE_FULL = 3 };

struct NormArgs {
    int T, D;
    int rt, yt, xt, wt;  // DT_F32 / DT_BF16 of the residual, the block output, x and the weights
    int gate;
    bool post, next;
    float eps_post, eps_next, alpha, beta;
    const void *w_post, *w_next;
    // forward
    const void *r, *y, *g;
    void *r_out, *x;
    float *rstd;  // [2][T]: rstd of y, rstd of r_out
    // backward (r_out and rstd are read)
    const void *dr_out, *dx;
    void *dr, *dy, *dg, *dw_post, *dw_next;
    float *part;  // [norm_parts(D)][3][D]
};

constexpr int kMaxNormWidth = 16384;
constexpr int kWaveWidth = 512;  // widest row of a single wave

// rows of partial column sums in the backward: its blocks, or its waves where each has a row
constexpr int norm_parts(int width) { return width <= kWaveWidth ? 4096 : 512; }

hipError_t launch_norm_forward(const NormArgs &a, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs &a, hipStream_t s);

// ---- AdamW (adamw.hip)
constexpr int kQBlock = 256;  // elements that share a scale of the 8-bit states

// One tensor in the device table.
struct AdamTensor {
    void *p;
    float *master;
    const void *g;
    void *m, *v;
    float *ms, *vs;
    int64_t n;
    float wd, lr_scale;
    uint8_t pt, gt, vec, pad;  // dtypes; vec: every pointer allows the wide loads
    uint32_t chunk0;           // first chunk of the tensor in the launch's chunk order
};
static_assert(sizeof(AdamTensor) == 80, "table layout");

struct AdamCtl {              // in the workspace, started by set_step
    unsigned long long step;  // steps taken
    // of the present step
    float clip;               // < 0: the step is skipped
    float lr, lr_m, root_v;   // lr, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
};

struct AdamArgs {
    const AdamTensor *tab;
    const uint32_t *chunk_of;  // [chunks] tensor of each chunk
    AdamCtl *ctl;
    double *part;              // [kAdamNormBlocks]
    int64_t chunks;
    int chunk_elems;           // elements of a chunk, a multiple of 1024
    bool e4m3, clipped;
    double beta1, beta2, lr;
    float eps, max_norm;
    const float *lr_dev;
    float *norm_out;
};

constexpr int kAdamNormBlocks = 2048;
constexpr int kAdamPut = 40;  // table entries per upload launch (3.2 KB of arguments)

struct AdamPut {
    AdamTensor t[kAdamPut];
};

hipError_t launch_adam_put(const AdamTensor *host, int n, AdamTensor *tab, hipStream_t s);
hipError_t launch_adam_map(const AdamTensor *tab, int n, uint32_t *chunk_of, int64_t chunks, hipStream_t s);
hipError_t launch_adam_set_step(AdamCtl *ctl, unsigned long long step, hipStream_t s);
hipError_t launch_adam_step(const AdamArgs &a, hipStream_t s);

// ---- gated feed-forward (ffn.hip)
constexpr int kFfnPlanes = 3;  // bf16 terms of an exactly carried fp32 operand

struct FfnArgs {
    int T, D, I, act;
    const uint16_t *wg, *wu, *wd;
    const uint16_t *x;
    // forward
    void *y;
    int yt;
    bool acc;
    float *gu;       // [T][2][I] or null
    // scratch
    uint16_t *h;     // [planes][T][I]
    uint16_t *dgu;   // [planes][T][2I]
    float *gu_ws;    // [T][2][I], used where saved_gu is missing
    float *part;     // parts of a reduction that is cut
    size_t part_floats;
    // backward
    const uint16_t *dy;
    const float *saved_gu;
    void *dx, *dwg, *dwu, *dwd;
    int dxt, dwt;
};

constexpr int kFewTokens = 64;  // most tokens of ffn_few.hip
hipError_t launch_ffn_few_gate_up(const FfnArgs &a, uint16_t *h, int planes, float *gu, hipStream_t s);
hipError_t launch_ffn_few_down(const FfnArgs &a, int planes, hipStream_t s);
hipError_t launch_ffn_forward(const FfnArgs &a, hipStream_t s);
hipError_t launch_ffn_backward(const FfnArgs &a, hipStream_t s);

}  // namespace moe
