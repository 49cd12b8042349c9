// block_api.hip -- the C ABI declared in include/moe_block.h: argument checks, workspace carving
// and kernel launches on the caller's stream.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <new>
#include <utility>
#include <vector>

#include "api_status.h"
#include "block_internal.h"
#include "common.h"
#include "moe_block.h"
#include "moe_internal.h"

using moe::api_fail;

namespace {

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

bool on(const void *p, size_t a) { return (uintptr_t)p % a == 0; }

size_t size_of(int32_t dt) { return dt == MOE_DT_F32 ? 4 : 2; }

bool is_dtype(int32_t dt) { return dt == MOE_DT_F32 || dt == MOE_DT_BF16; }

moe_status device_status(hipError_t e, const char *where)
{
    return e == hipSuccess ? MOE_OK : api_fail(MOE_ERR_DEVICE, "%s: %s", where, hipGetErrorString(e));
}

moe_status check_workspace(const void *ws, size_t have, size_t need)
{
    if (need == 0) return MOE_OK;
    if (!ws) return api_fail(MOE_ERR_WORKSPACE, "workspace is NULL");
    if (have < need) return api_fail(MOE_ERR_WORKSPACE, "workspace %zu bytes < required %zu", have, need);
    if (!on(ws, 256)) return api_fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    return MOE_OK;
}

moe_status check_T(int32_t T, int32_t most)
{
    if (T < 0 || T > most) return api_fail(MOE_ERR_INVALID_ARG, "T=%d must be in 0..max_tokens=%d", T, most);
    return MOE_OK;
}

struct Buf {
    const void *p;
    size_t bytes;
    const char *name;
};

// No output may share memory with another output or with an input.
moe_status check_overlap(std::initializer_list<Buf> outs, std::initializer_list<Buf> ins)
{
    auto hit = [](const Buf &a, const Buf &b) {
        return a.p && b.p && (uintptr_t)a.p < (uintptr_t)b.p + b.bytes && (uintptr_t)b.p < (uintptr_t)a.p + a.bytes;
    };
    for (const Buf *a = outs.begin(); a != outs.end(); a++) {
        for (const Buf *b = a + 1; b != outs.end(); b++)
            if (hit(*a, *b)) return api_fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", a->name, b->name);
        for (const Buf &b : ins)
            if (hit(*a, b)) return api_fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", a->name, b.name);
    }
    return MOE_OK;
}

// ---------------------------------------------------------------- gated feed-forward

constexpr int kMaxFfnWidth = 1 << 20;

struct FfnLayout {
    size_t h, dgu, gu, part, part_floats, total;
};

// Floats for the parts of a cut reduction: sixteen parts of the largest output, at most 64 MB.
constexpr size_t kPartFloats = (size_t)16 << 20;

FfnLayout ffn_layout(const moe_ffn_desc &d)
{
    const size_t T = d.max_tokens, I = d.inter;
    const bool back = (d.flags & MOE_FFN_BACKWARD) != 0;
    FfnLayout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += up256(bytes);
        return at;
    };
    L.h = take(moe::kFfnPlanes * T * I * 2);
    L.dgu = take(back ? moe::kFfnPlanes * T * 2 * I * 2 : 0);
    L.gu = take(back ? T * 2 * I * 4 : 0);
    const size_t D = d.width, most = std::max({T * 2 * I, T * D, back ? 3 * D * I : 0});
    L.part_floats = std::min(16 * most, kPartFloats);
    L.part = take(L.part_floats * 4);
    L.total = off;
    return L;
}

moe_status check_ffn_desc(const moe_ffn_desc *d)
{
    if (!d) return api_fail(MOE_ERR_INVALID_ARG, "desc is NULL");
    if (d->width <= 0 || d->width % 8 || d->width > kMaxFfnWidth)
        return api_fail(MOE_ERR_INVALID_ARG, "width=%d must be a positive multiple of 8, at most %d", d->width, kMaxFfnWidth);
    if (d->inter <= 0 || d->inter % 8 || d->inter > kMaxFfnWidth)
        return api_fail(MOE_ERR_INVALID_ARG, "inter=%d must be a positive multiple of 8, at most %d", d->inter, kMaxFfnWidth);
    if (d->max_tokens < 0 || d->max_tokens > (1 << 24))
        return api_fail(MOE_ERR_INVALID_ARG, "max_tokens=%d must be in 0..2^24", d->max_tokens);
    if (d->act != MOE_ACT_SWIGLU && d->act != MOE_ACT_SITU)
        return api_fail(MOE_ERR_UNSUPPORTED, "activation %d is not implemented", d->act);
    if (d->flags & ~(uint32_t)MOE_FFN_BACKWARD) return api_fail(MOE_ERR_INVALID_ARG, "unknown flags 0x%x", d->flags);
    return MOE_OK;
}

// ---------------------------------------------------------------- block norms

moe_status check_norm_desc(const moe_norm_desc *d)
{
    if (!d) return api_fail(MOE_ERR_INVALID_ARG, "desc is NULL");
    if (d->width <= 0 || d->width > moe::kMaxNormWidth)
        return api_fail(MOE_ERR_INVALID_ARG, "width=%d must be in 1..%d", d->width, moe::kMaxNormWidth);
    if (d->max_tokens < 0 || d->max_tokens > (1 << 30)) return api_fail(MOE_ERR_INVALID_ARG, "max_tokens=%d must be in 0..2^30", d->max_tokens);
    if (!is_dtype(d->r_dtype) || !is_dtype(d->y_dtype) || !is_dtype(d->x_dtype) || !is_dtype(d->w_dtype))
        return api_fail(MOE_ERR_INVALID_ARG, "a dtype (r %d, y %d, x %d, w %d) is not f32/bf16", d->r_dtype, d->y_dtype,
                        d->x_dtype, d->w_dtype);
    if (d->gate < MOE_GATE_NONE || d->gate > MOE_GATE_FULL) return api_fail(MOE_ERR_INVALID_ARG, "unknown gate %d", d->gate);
    if (!(d->eps_post > 0.f) || !(d->eps_next > 0.f) || !std::isfinite(d->eps_post) || !std::isfinite(d->eps_next))
        return api_fail(MOE_ERR_INVALID_ARG, "eps_post=%g and eps_next=%g must be positive and finite", d->eps_post, d->eps_next);
    if (!std::isfinite(d->res_scale) || !std::isfinite(d->branch_scale))
        return api_fail(MOE_ERR_INVALID_ARG, "res_scale or branch_scale is not finite");
    if (d->flags & ~(uint32_t)(MOE_NORM_POST | MOE_NORM_NEXT | MOE_NORM_BACKWARD))
        return api_fail(MOE_ERR_INVALID_ARG, "unknown flags 0x%x", d->flags);
    return MOE_OK;
}

size_t norm_bytes(const moe_norm_desc &d)
{
    if (!(d.flags & MOE_NORM_BACKWARD)) return 0;
    return up256((size_t)std::min(d.max_tokens, moe::norm_parts(d.width)) * 3 * d.width * 4);
}

// ---------------------------------------------------------------- AdamW

constexpr int kChunk = 1024;  // smallest chunk: an iteration of a block

struct AdamLayout {
    size_t ctl, part, tab, map, total;
};

// chunk size for this many elements: small sets are spread over many blocks, large ones do more per block
int chunk_for(int64_t elements) { return elements < ((int64_t)1 << 22) ? kChunk : 4 * kChunk; }

// most chunks that max_tensors tensors of max_elements elements in all can have: the part of a chunk
// that each tensor's end leaves empty counts once for each tensor
int64_t most_chunks(const moe_adamw_desc &d)
{
    const int64_t small = std::min<int64_t>(d.max_elements, (int64_t)1 << 22) / kChunk;
    return std::max(small, d.max_elements / (4 * kChunk)) + d.max_tensors;
}

AdamLayout adam_layout(const moe_adamw_desc &d)
{
    AdamLayout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += up256(bytes);
        return at;
    };
    L.ctl = take(sizeof(moe::AdamCtl));
    L.part = take((size_t)moe::kAdamNormBlocks * 8);
    L.tab = take((size_t)d.max_tensors * sizeof(moe::AdamTensor));
    L.map = take((size_t)most_chunks(d) * 4);
    L.total = off;
    return L;
}

moe_status check_adam_desc(const moe_adamw_desc *d)
{
    if (!d) return api_fail(MOE_ERR_INVALID_ARG, "desc is NULL");
    if (!(d->beta1 >= 0 && d->beta1 < 1) || !(d->beta2 >= 0 && d->beta2 < 1))
        return api_fail(MOE_ERR_INVALID_ARG, "beta1=%g and beta2=%g must be in [0, 1)", d->beta1, d->beta2);
    if (!((float)d->eps > 0.f) || !std::isfinite((float)d->eps))
        return api_fail(MOE_ERR_INVALID_ARG, "eps=%g must be positive and finite in fp32", d->eps);
    if (!(d->max_norm >= 0) || !std::isfinite((float)d->max_norm) || (d->max_norm > 0 && !((float)d->max_norm > 0.f)))
        return api_fail(MOE_ERR_INVALID_ARG, "max_norm=%g must be 0 or positive and finite in fp32", d->max_norm);
    if (d->state != MOE_STATE_F32 && d->state != MOE_STATE_E4M3)
        return api_fail(MOE_ERR_INVALID_ARG, "unknown state format %d", d->state);
    if (d->max_tensors < 1 || d->max_tensors > (1 << 20))
        return api_fail(MOE_ERR_INVALID_ARG, "max_tensors=%d must be in 1..2^20", d->max_tensors);
    if (d->max_elements < 0 || d->max_elements > ((int64_t)1 << 40))
        return api_fail(MOE_ERR_INVALID_ARG, "max_elements=%lld must be in 0..2^40", (long long)d->max_elements);
    return MOE_OK;
}

}  // namespace

struct moe_ffn {
    moe_ffn_desc d;
    const uint16_t *wg, *wu, *wd;
    char *ws;
    FfnLayout lay;
};

struct moe_norm {
    moe_norm_desc d;
    const void *w_post, *w_next;
    float *part;
};

struct moe_adamw {
    moe_adamw_desc d;
    char *ws;
    AdamLayout lay;
    bool bound = false, counted = false;
    int64_t chunks = 0;
    int chunk_elems = kChunk;
    // the bytes that a step reads or writes, in address order and disjoint: the bound buffers and the workspace
    std::vector<std::pair<uintptr_t, uintptr_t>> used;

    bool uses(const void *p, size_t bytes) const
    {
        const uintptr_t lo = (uintptr_t)p, hi = lo + bytes;
        const auto i = std::upper_bound(used.begin(), used.end(), lo, [](uintptr_t v, const auto &r) { return v < r.second; });
        return p && i != used.end() && i->first < hi;
    }
};

namespace {

moe::FfnArgs ffn_args(const moe_ffn *f, const uint16_t *x, int32_t T)
{
    moe::FfnArgs a{};
    a.T = T, a.D = f->d.width, a.I = f->d.inter, a.act = f->d.act;
    a.wg = f->wg, a.wu = f->wu, a.wd = f->wd, a.x = x;
    a.h = (uint16_t *)(f->ws + f->lay.h);
    a.dgu = (uint16_t *)(f->ws + f->lay.dgu);
    a.gu_ws = (float *)(f->ws + f->lay.gu);
    a.part = (float *)(f->ws + f->lay.part);
    a.part_floats = f->lay.part_floats;
    return a;
}

moe::NormArgs norm_args(const moe_norm *h, int32_t T)
{
    moe::NormArgs a{};
    const moe_norm_desc &d = h->d;
    a.T = T, a.D = d.width;
    a.rt = d.r_dtype, a.yt = d.y_dtype, a.xt = d.x_dtype, a.wt = d.w_dtype;
    a.gate = d.gate;
    a.post = (d.flags & MOE_NORM_POST) != 0, a.next = (d.flags & MOE_NORM_NEXT) != 0;
    a.eps_post = d.eps_post, a.eps_next = d.eps_next, a.alpha = d.res_scale, a.beta = d.branch_scale;
    a.w_post = h->w_post, a.w_next = h->w_next;
    a.part = h->part;
    return a;
}

// the gate's argument against the descriptor, with y or without it
moe_status check_gate(const moe_norm *h, const void *y, const void *gate)
{
    const bool wants = y && h->d.gate != MOE_GATE_NONE;
    if (wants != (gate != nullptr))
        return api_fail(MOE_ERR_INVALID_ARG, wants ? "gate is NULL" : "gate must be NULL (no gate, or no y)");
    if (gate && !on(gate, h->d.gate == MOE_GATE_FULL ? size_of(h->d.y_dtype) : 4))
        return api_fail(MOE_ERR_INVALID_ARG, "gate is not aligned to its element");
    return MOE_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- gated feed-forward

void moe_ffn_desc_init(moe_ffn_desc *d)
{
    if (!d) return;
    *d = moe_ffn_desc{};
    d->width = 3584;
    d->inter = 6144;
    d->max_tokens = 4096;
    d->act = MOE_ACT_SWIGLU;
    d->flags = MOE_FFN_BACKWARD;
}

moe_status moe_ffn_workspace_size(const moe_ffn_desc *d, size_t *bytes)
{
    moe::api_clear();
    moe_status st = check_ffn_desc(d);
    if (st != MOE_OK) return st;
    if (!bytes) return api_fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = ffn_layout(*d).total;
    return MOE_OK;
}

moe_status moe_ffn_create(const moe_ffn_desc *d, const uint16_t *w_gate, const uint16_t *w_up, const uint16_t *w_down,
                          void *workspace, size_t ws_bytes, moe_ffn **out)
{
    moe::api_clear();
    moe_status st = check_ffn_desc(d);
    if (st != MOE_OK) return st;
    if (!out) return api_fail(MOE_ERR_INVALID_ARG, "out is NULL");
    if (!w_gate || !w_up || !w_down) return api_fail(MOE_ERR_INVALID_ARG, "a weight is NULL");
    if (!on(w_gate, 16) || !on(w_up, 16) || !on(w_down, 16))
        return api_fail(MOE_ERR_INVALID_ARG, "the weights must be 16-byte aligned");
    const FfnLayout lay = ffn_layout(*d);
    if ((st = check_workspace(workspace, ws_bytes, lay.total)) != MOE_OK) return st;
    moe_ffn *f = new (std::nothrow) moe_ffn{*d, w_gate, w_up, w_down, (char *)workspace, lay};
    if (!f) return api_fail(MOE_ERR_INTERNAL, "out of host memory");
    *out = f;
    return MOE_OK;
}

moe_status moe_ffn_forward(moe_ffn *f, const uint16_t *x, int32_t T, void *y, int32_t yt, int32_t accumulate,
                           float *saved_gu, void *stream)
{
    moe::api_clear();
    moe_status st;
    if (!f) return api_fail(MOE_ERR_INVALID_ARG, "handle is NULL");
    if ((st = check_T(T, f->d.max_tokens)) != MOE_OK) return st;
    if (!is_dtype(yt)) return api_fail(MOE_ERR_INVALID_ARG, "y dtype %d is not f32/bf16", yt);
    if (T == 0) return MOE_OK;
    if (!x || !y) return api_fail(MOE_ERR_INVALID_ARG, "x or y is NULL");
    if (!on(x, 16) || !on(y, 16) || !on(saved_gu, 16))
        return api_fail(MOE_ERR_INVALID_ARG, "x, y and saved_gu must be 16-byte aligned");
    const size_t TD = (size_t)T * f->d.width, DI = (size_t)f->d.width * f->d.inter, TI = (size_t)T * f->d.inter;
    if ((st = check_overlap({{y, TD * size_of(yt), "y"}, {saved_gu, TI * 8, "saved_gu"}, {f->ws, f->lay.total, "the workspace"}},
                            {{x, TD * 2, "x"}, {f->wg, DI * 2, "w_gate"}, {f->wu, DI * 2, "w_up"}, {f->wd, DI * 2, "w_down"}})) != MOE_OK)
        return st;
    moe::FfnArgs a = ffn_args(f, x, T);
    a.y = y, a.yt = yt, a.acc = accumulate != 0, a.gu = saved_gu;
    return device_status(moe::launch_ffn_forward(a, (hipStream_t)stream), "feed-forward");
}

moe_status moe_ffn_backward(moe_ffn *f, const uint16_t *x, const uint16_t *dy, int32_t T, const float *saved_gu,
                            void *dx, int32_t dxt, int32_t accumulate, void *dw_gate, void *dw_up, void *dw_down,
                            int32_t dwt, void *stream)
{
    moe::api_clear();
    moe_status st;
    if (!f) return api_fail(MOE_ERR_INVALID_ARG, "handle is NULL");
    if (!(f->d.flags & MOE_FFN_BACKWARD)) return api_fail(MOE_ERR_INVALID_ARG, "the workspace was sized without MOE_FFN_BACKWARD");
    if ((st = check_T(T, f->d.max_tokens)) != MOE_OK) return st;
    if (!is_dtype(dxt) || !is_dtype(dwt)) return api_fail(MOE_ERR_INVALID_ARG, "a gradient dtype (%d, %d) is not f32/bf16", dxt, dwt);
    if (!on(x, 16) || !on(dy, 16) || !on(saved_gu, 16) || !on(dx, 16) || !on(dw_gate, 16) || !on(dw_up, 16) || !on(dw_down, 16))
        return api_fail(MOE_ERR_INVALID_ARG, "x, dy, saved_gu and the gradients must be 16-byte aligned");
    const hipStream_t s = (hipStream_t)stream;
    if (T == 0) {
        const size_t n = (size_t)f->d.width * f->d.inter * size_of(dwt) / 4;
        for (void *w : {dw_gate, dw_up, dw_down}) {
            if (!w) continue;
            if ((st = device_status(moe::fill_zero((float *)w, n, s), "zero weight gradients")) != MOE_OK) return st;
        }
        return MOE_OK;
    }
    if (!x || !dy) return api_fail(MOE_ERR_INVALID_ARG, "x or dy is NULL");
    if (!dx && !dw_gate && !dw_up && !dw_down) return MOE_OK;
    const size_t TD = (size_t)T * f->d.width, DI = (size_t)f->d.width * f->d.inter, TI = (size_t)T * f->d.inter, wb = DI * size_of(dwt);
    if ((st = check_overlap({{dx, TD * size_of(dxt), "dx"}, {dw_gate, wb, "dw_gate"}, {dw_up, wb, "dw_up"}, {dw_down, wb, "dw_down"}, {f->ws, f->lay.total, "the workspace"}},
                            {{x, TD * 2, "x"}, {dy, TD * 2, "dy"}, {saved_gu, TI * 8, "saved_gu"}, {f->wg, DI * 2, "w_gate"}, {f->wu, DI * 2, "w_up"}, {f->wd, DI * 2, "w_down"}})) != MOE_OK)
        return st;
    moe::FfnArgs a = ffn_args(f, x, T);
    a.dy = dy, a.saved_gu = saved_gu, a.dx = dx, a.dxt = dxt, a.acc = accumulate != 0;
    a.dwg = dw_gate, a.dwu = dw_up, a.dwd = dw_down, a.dwt = dwt;
    return device_status(moe::launch_ffn_backward(a, s), "feed-forward gradients");
}

void moe_ffn_destroy(moe_ffn *f) { delete f; }

// ---------------------------------------------------------------- block norms

void moe_norm_desc_init(moe_norm_desc *d)
{
    if (!d) return;
    *d = moe_norm_desc{};
    d->width = 3584;
    d->max_tokens = 4096;
    d->r_dtype = d->y_dtype = d->w_dtype = MOE_DT_F32;
    d->x_dtype = MOE_DT_BF16;
    d->gate = MOE_GATE_NONE;
    d->eps_post = d->eps_next = 1e-6f;
    d->res_scale = d->branch_scale = 1.f;
    d->flags = MOE_NORM_POST | MOE_NORM_NEXT | MOE_NORM_BACKWARD;
}

moe_status moe_norm_workspace_size(const moe_norm_desc *d, size_t *bytes)
{
    moe::api_clear();
    moe_status st = check_norm_desc(d);
    if (st != MOE_OK) return st;
    if (!bytes) return api_fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = norm_bytes(*d);
    return MOE_OK;
}

moe_status moe_norm_create(const moe_norm_desc *d, const void *w_post, const void *w_next, void *workspace,
                           size_t ws_bytes, moe_norm **out)
{
    moe::api_clear();
    moe_status st = check_norm_desc(d);
    if (st != MOE_OK) return st;
    if (!out) return api_fail(MOE_ERR_INVALID_ARG, "out is NULL");
    const bool post = (d->flags & MOE_NORM_POST) != 0, next = (d->flags & MOE_NORM_NEXT) != 0;
    if (post != (w_post != nullptr)) return api_fail(MOE_ERR_INVALID_ARG, post ? "w_post is NULL" : "w_post without MOE_NORM_POST");
    if (next != (w_next != nullptr)) return api_fail(MOE_ERR_INVALID_ARG, next ? "w_next is NULL" : "w_next without MOE_NORM_NEXT");
    if (!on(w_post, size_of(d->w_dtype)) || !on(w_next, size_of(d->w_dtype)))
        return api_fail(MOE_ERR_INVALID_ARG, "w_post and w_next must be aligned to their element");
    if ((st = check_workspace(workspace, ws_bytes, norm_bytes(*d))) != MOE_OK) return st;
    moe_norm *h = new (std::nothrow) moe_norm{*d, w_post, w_next, (float *)workspace};
    if (!h) return api_fail(MOE_ERR_INTERNAL, "out of host memory");
    *out = h;
    return MOE_OK;
}

moe_status moe_norm_forward(moe_norm *h, const void *r, const void *y, const void *gate, int32_t T, void *r_out,
                            void *x, float *rstd, void *stream)
{
    moe::api_clear();
    moe_status st;
    if (!h) return api_fail(MOE_ERR_INVALID_ARG, "handle is NULL");
    if ((st = check_T(T, h->d.max_tokens)) != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    const bool next = (h->d.flags & MOE_NORM_NEXT) != 0;
    if (!r) return api_fail(MOE_ERR_INVALID_ARG, "r is NULL");
    if ((y != nullptr) != (r_out != nullptr)) return api_fail(MOE_ERR_INVALID_ARG, y ? "r_out is NULL" : "r_out must be NULL without y");
    if (next != (x != nullptr)) return api_fail(MOE_ERR_INVALID_ARG, next ? "x is NULL" : "x must be NULL without MOE_NORM_NEXT");
    if (!y && !next) return api_fail(MOE_ERR_INVALID_ARG, "nothing to compute: no y and no MOE_NORM_NEXT");
    if ((st = check_gate(h, y, gate)) != MOE_OK) return st;
    if (!on(r, size_of(h->d.r_dtype)) || !on(r_out, size_of(h->d.r_dtype)) || !on(y, size_of(h->d.y_dtype)) ||
        !on(x, size_of(h->d.x_dtype)) || !on(rstd, 4))
        return api_fail(MOE_ERR_INVALID_ARG, "a buffer is not aligned to its element");
    const size_t D = h->d.width, TD = (size_t)T * D, rb = TD * size_of(h->d.r_dtype), wb = D * size_of(h->d.w_dtype);
    const Buf g = {gate, h->d.gate == MOE_GATE_FULL ? TD * size_of(h->d.y_dtype) : 4 * (h->d.gate == MOE_GATE_TOKEN ? (size_t)T : D), "gate"};
    if ((st = check_overlap({{r_out, rb, "r_out"}, {x, TD * size_of(h->d.x_dtype), "x"}, {rstd, (size_t)T * 8, "rstd"}},
                            {{r == r_out ? nullptr : r, rb, "r"}, {y, TD * size_of(h->d.y_dtype), "y"}, g, {h->w_post, wb, "w_post"}, {h->w_next, wb, "w_next"}})) != MOE_OK)
        return st;
    moe::NormArgs a = norm_args(h, T);
    a.r = r, a.y = y, a.g = gate, a.r_out = r_out, a.x = x, a.rstd = rstd;
    return device_status(moe::launch_norm_forward(a, (hipStream_t)stream), "block norm");
}

moe_status moe_norm_backward(moe_norm *h, const void *y, const void *gate, const void *r_out, const float *rstd,
                             const void *dr_out, const void *dx, int32_t T, void *dr, void *dy, void *dgate,
                             void *dw_post, void *dw_next, void *stream)
{
    moe::api_clear();
    moe_status st;
    if (!h) return api_fail(MOE_ERR_INVALID_ARG, "handle is NULL");
    const moe_norm_desc &d = h->d;
    const bool post = (d.flags & MOE_NORM_POST) != 0, next = (d.flags & MOE_NORM_NEXT) != 0;
    if (!(d.flags & MOE_NORM_BACKWARD)) return api_fail(MOE_ERR_INVALID_ARG, "the workspace was sized without MOE_NORM_BACKWARD");
    if ((st = check_T(T, d.max_tokens)) != MOE_OK) return st;
    if (dw_post && !post) return api_fail(MOE_ERR_INVALID_ARG, "dw_post without MOE_NORM_POST");
    if (dw_next && !next) return api_fail(MOE_ERR_INVALID_ARG, "dw_next without MOE_NORM_NEXT");
    if (dgate && d.gate == MOE_GATE_NONE) return api_fail(MOE_ERR_INVALID_ARG, "dgate without a gate");
    const size_t gs = d.gate == MOE_GATE_FULL ? size_of(d.y_dtype) : 4, ws = size_of(d.w_dtype);
    if (!on(dw_post, ws) || !on(dw_next, ws) || !on(dgate, gs))
        return api_fail(MOE_ERR_INVALID_ARG, "dw_post, dw_next or dgate is not aligned to its element");
    if (T > 0) {
        if (!dr) return api_fail(MOE_ERR_INVALID_ARG, "dr is NULL");
        if (next != (dx != nullptr)) return api_fail(MOE_ERR_INVALID_ARG, next ? "dx is NULL" : "dx must be NULL without MOE_NORM_NEXT");
        if (next && !r_out) return api_fail(MOE_ERR_INVALID_ARG, "r_out is NULL");
        if (!rstd && (next || (post && y))) return api_fail(MOE_ERR_INVALID_ARG, "rstd is NULL");
        if ((y != nullptr) != (dy != nullptr)) return api_fail(MOE_ERR_INVALID_ARG, y ? "dy is NULL" : "dy must be NULL without y");
        if (!y && !next) return api_fail(MOE_ERR_INVALID_ARG, "nothing to compute: no y and no MOE_NORM_NEXT");
        if (!y && (dgate || dw_post)) return api_fail(MOE_ERR_INVALID_ARG, "dgate and dw_post need y");
        if ((st = check_gate(h, y, gate)) != MOE_OK) return st;
        const size_t rs = size_of(d.r_dtype), ys = size_of(d.y_dtype);
        if (!on(r_out, rs) || !on(dr_out, rs) || !on(dr, rs) || !on(y, ys) || !on(dy, ys) || !on(dx, size_of(d.x_dtype)) || !on(rstd, 4))
            return api_fail(MOE_ERR_INVALID_ARG, "a buffer is not aligned to its element");
        const size_t D = d.width, TD = (size_t)T * D, gb = d.gate == MOE_GATE_FULL ? TD * ys : 4 * (d.gate == MOE_GATE_TOKEN ? (size_t)T : D);
        if ((st = check_overlap({{dr, TD * rs, "dr"}, {dy, TD * ys, "dy"}, {dgate, gb, "dgate"}, {dw_post, D * ws, "dw_post"}, {dw_next, D * ws, "dw_next"},
                                 {h->part, norm_bytes(d), "the workspace"}},
                                {{dr == dr_out ? nullptr : dr_out, TD * rs, "dr_out"}, {r_out, TD * rs, "r_out"}, {y, TD * ys, "y"}, {gate, gb, "gate"},
                                 {dx, TD * size_of(d.x_dtype), "dx"}, {rstd, (size_t)T * 8, "rstd"}, {h->w_post, D * ws, "w_post"}, {h->w_next, D * ws, "w_next"}})) != MOE_OK)
            return st;
    }
    moe::NormArgs a = norm_args(h, T);
    a.y = y, a.g = gate, a.r_out = const_cast<void *>(r_out), a.rstd = const_cast<float *>(rstd);
    a.dr_out = dr_out, a.dx = dx, a.dr = dr, a.dy = dy, a.dg = dgate, a.dw_post = dw_post, a.dw_next = dw_next;
    return device_status(moe::launch_norm_backward(a, (hipStream_t)stream), "block norm gradients");
}

void moe_norm_destroy(moe_norm *h) { delete h; }

// ---------------------------------------------------------------- AdamW

void moe_adamw_desc_init(moe_adamw_desc *d)
{
    if (!d) return;
    *d = moe_adamw_desc{};
    d->beta1 = 0.9;
    d->beta2 = 0.999;
    d->eps = 1e-8;
    d->state = MOE_STATE_F32;
    d->max_tensors = 1024;
    d->max_elements = (int64_t)1 << 28;
}

moe_status moe_adamw_workspace_size(const moe_adamw_desc *d, size_t *bytes)
{
    moe::api_clear();
    moe_status st = check_adam_desc(d);
    if (st != MOE_OK) return st;
    if (!bytes) return api_fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = adam_layout(*d).total;
    return MOE_OK;
}

moe_status moe_adamw_create(const moe_adamw_desc *d, void *workspace, size_t ws_bytes, moe_adamw **out)
{
    moe::api_clear();
    moe_status st = check_adam_desc(d);
    if (st != MOE_OK) return st;
    if (!out) return api_fail(MOE_ERR_INVALID_ARG, "out is NULL");
    const AdamLayout lay = adam_layout(*d);
    if ((st = check_workspace(workspace, ws_bytes, lay.total)) != MOE_OK) return st;
    moe_adamw *a = new (std::nothrow) moe_adamw{*d, (char *)workspace, lay};
    if (!a) return api_fail(MOE_ERR_INTERNAL, "out of host memory");
    *out = a;
    return MOE_OK;
}

moe_status moe_adamw_bind(moe_adamw *a, const moe_adamw_tensor *t, int32_t n, void *stream)
try {
    moe::api_clear();
    if (!a) return api_fail(MOE_ERR_INVALID_ARG, "handle is NULL");
    if (n < 0 || n > a->d.max_tensors) return api_fail(MOE_ERR_INVALID_ARG, "n=%d must be in 0..max_tensors=%d", n, a->d.max_tensors);
    if (n > 0 && !t) return api_fail(MOE_ERR_INVALID_ARG, "tensors is NULL");
    const bool small = a->d.state == MOE_STATE_E4M3;
    struct Range {
        uintptr_t lo, hi;
        bool written;
        int tensor;
    };
    std::vector<Range> ranges;
    std::vector<moe::AdamTensor> tab;
    int64_t total = 0;
    for (int i = 0; i < n; i++) {
        const moe_adamw_tensor &e = t[i];
        if (e.n < 0) return api_fail(MOE_ERR_INVALID_ARG, "tensor %d: n=%lld is negative", i, (long long)e.n);
        if (!is_dtype(e.param_dtype) || !is_dtype(e.grad_dtype)) return api_fail(MOE_ERR_INVALID_ARG, "tensor %d: a dtype is not f32/bf16", i);
        if (!std::isfinite(e.weight_decay) || !std::isfinite(e.lr_scale))
            return api_fail(MOE_ERR_INVALID_ARG, "tensor %d: weight_decay or lr_scale is not finite", i);
        if (e.n == 0) continue;
        if (e.n > a->d.max_elements - total) return api_fail(MOE_ERR_INVALID_ARG, "more than max_elements=%lld elements", (long long)a->d.max_elements);
        total += e.n;
        if (!e.param || !e.grad || !e.m || !e.v) return api_fail(MOE_ERR_INVALID_ARG, "tensor %d: param, grad, m or v is NULL", i);
        if (small != (e.m_scale != nullptr) || small != (e.v_scale != nullptr))
            return api_fail(MOE_ERR_INVALID_ARG, small ? "tensor %d: m_scale or v_scale is NULL" : "tensor %d: scales without MOE_STATE_E4M3", i);
        const size_t ss = small ? 1 : 4, ps = size_of(e.param_dtype), gs = size_of(e.grad_dtype);
        if (!on(e.param, ps) || !on(e.grad, gs) || !on(e.master, 4) || !on(e.m, ss) || !on(e.v, ss) || !on(e.m_scale, 4) || !on(e.v_scale, 4))
            return api_fail(MOE_ERR_INVALID_ARG, "tensor %d: a buffer is not aligned to its element", i);
        const size_t nq = (size_t)((e.n + moe::kQBlock - 1) / moe::kQBlock);
        auto add = [&](const void *p, size_t bytes, bool written) {
            if (p) ranges.push_back({(uintptr_t)p, (uintptr_t)p + bytes, written, i});
        };
        add(e.param, e.n * ps, true);
        add(e.master, e.n * 4, true);
        add(e.m, e.n * ss, true);
        add(e.v, e.n * ss, true);
        add(e.m_scale, nq * 4, true);
        add(e.v_scale, nq * 4, true);
        add(e.grad, e.n * gs, false);
        // loads and stores of four elements: 16 bytes of fp32, 8 of bf16, 4 of codes
        const bool vec = on(e.param, 4 * ps) && on(e.grad, 4 * gs) && on(e.master, 16) && on(e.m, 4 * ss) && on(e.v, 4 * ss);
        tab.push_back({e.param, e.master, e.grad, e.m, e.v, e.m_scale, e.v_scale, e.n, e.weight_decay, e.lr_scale,
                       (uint8_t)e.param_dtype, (uint8_t)e.grad_dtype, (uint8_t)vec, 0, 0});
    }
    // in address order every range has to begin at or behind the end of what is written before it, and a
    // written one behind the end of everything before it
    ranges.push_back({(uintptr_t)a->ws, (uintptr_t)a->ws + a->lay.total, true, -1});
    std::sort(ranges.begin(), ranges.end(), [](const Range &x, const Range &y) { return x.lo < y.lo; });
    uintptr_t end = 0, end_written = 0;
    int last = -1;  // whose range ends at end
    std::vector<std::pair<uintptr_t, uintptr_t>> used;
    for (const Range &r : ranges) {
        if (r.lo < (r.written ? end : end_written))
            return api_fail(MOE_ERR_INVALID_ARG, "tensor %d: a buffer overlaps one that the step writes (a tensor's or the workspace)",
                            r.tensor < 0 ? last : r.tensor);
        if (used.empty() || r.lo > end)
            used.push_back({r.lo, r.hi});
        else
            used.back().second = std::max(end, r.hi);
        if (r.hi > end) end = r.hi, last = r.tensor;
        if (r.written) end_written = std::max(end_written, r.hi);
    }
    const int ce = chunk_for(total);
    int64_t chunks = 0;
    for (moe::AdamTensor &e : tab) {
        e.chunk0 = (uint32_t)chunks;
        chunks += (e.n + ce - 1) / ce;
    }
    const hipStream_t s = (hipStream_t)stream;
    moe::AdamTensor *dev = (moe::AdamTensor *)(a->ws + a->lay.tab);
    a->bound = false;
    hipError_t e = moe::launch_adam_put(tab.data(), (int)tab.size(), dev, s);
    if (e == hipSuccess) e = moe::launch_adam_map(dev, (int)tab.size(), (uint32_t *)(a->ws + a->lay.map), chunks, s);
    if (e != hipSuccess) return device_status(e, "tensor table");
    a->bound = true;
    a->chunks = chunks;
    a->chunk_elems = ce;
    a->used.swap(used);
    return MOE_OK;
} catch (...) {
    return MOE_ERR_INTERNAL;  // out of host memory: no text, which would need some
}

moe_status moe_adamw_set_step(moe_adamw *a, int64_t steps, void *stream)
{
    moe::api_clear();
    if (!a) return api_fail(MOE_ERR_INVALID_ARG, "handle is NULL");
    if (steps < 0) return api_fail(MOE_ERR_INVALID_ARG, "steps=%lld is negative", (long long)steps);
    const moe_status st = device_status(moe::launch_adam_set_step((moe::AdamCtl *)(a->ws + a->lay.ctl), (unsigned long long)steps, (hipStream_t)stream),
                                        "step count");
    if (st == MOE_OK) a->counted = true;
    return st;
}

moe_status moe_adamw_step(moe_adamw *a, double lr, const float *lr_dev, float *grad_norm, void *stream)
{
    moe::api_clear();
    if (!a) return api_fail(MOE_ERR_INVALID_ARG, "handle is NULL");
    if (!a->bound) return api_fail(MOE_ERR_INVALID_ARG, "no tensors are bound (moe_adamw_bind)");
    if (!a->counted) return api_fail(MOE_ERR_INVALID_ARG, "the step count is not set (moe_adamw_set_step)");
    if (!lr_dev && !std::isfinite(lr)) return api_fail(MOE_ERR_INVALID_ARG, "lr=%g is not finite", lr);
    if (!on(lr_dev, 4) || !on(grad_norm, 4)) return api_fail(MOE_ERR_INVALID_ARG, "lr_dev or grad_norm is not aligned to its element");
    if (grad_norm && !(a->d.max_norm > 0)) return api_fail(MOE_ERR_INVALID_ARG, "grad_norm needs max_norm > 0");
    if (a->uses(grad_norm, 4)) return api_fail(MOE_ERR_INVALID_ARG, "grad_norm overlaps a bound tensor or the workspace");
    if (lr_dev && grad_norm && (uintptr_t)lr_dev < (uintptr_t)grad_norm + 4 && (uintptr_t)grad_norm < (uintptr_t)lr_dev + 4)
        return api_fail(MOE_ERR_INVALID_ARG, "grad_norm overlaps lr_dev");
    moe::AdamArgs s{};
    s.tab = (const moe::AdamTensor *)(a->ws + a->lay.tab);
    s.chunk_of = (const uint32_t *)(a->ws + a->lay.map);
    s.ctl = (moe::AdamCtl *)(a->ws + a->lay.ctl);
    s.part = (double *)(a->ws + a->lay.part);
    s.chunks = a->chunks, s.chunk_elems = a->chunk_elems;
    s.e4m3 = a->d.state == MOE_STATE_E4M3;
    s.clipped = a->d.max_norm > 0;
    s.beta1 = a->d.beta1, s.beta2 = a->d.beta2, s.lr = lr;
    s.eps = (float)a->d.eps, s.max_norm = (float)a->d.max_norm;
    s.lr_dev = lr_dev, s.norm_out = grad_norm;
    return device_status(moe::launch_adam_step(s, (hipStream_t)stream), "AdamW step");
}

void moe_adamw_destroy(moe_adamw *a) { delete a; }

}  // extern "C"
