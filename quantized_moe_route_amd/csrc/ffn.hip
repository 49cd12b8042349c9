// ffn.hip -- the dense gated feed-forward block (include/moe_block.h has the formulas).
//
// Five products, all C[m][n] = sum_k A(m, k) B(n, k) in bf16 with fp32 accumulation:
//   gate/up   A = x [T][D],          B = Wg, Wu [I][D]      epilogue: act, h (and g, u)
//   down      A = h [T][I],          B = Wd [D][I]          epilogue: y
//   d h       A = dy [T][D],         B = Wd [D][I] by k     epilogue: act', dg, du, h
//   d x       A = dg | du [T][2I],   B = Wg, Wu [I][D] by k epilogue: dx
//   d W       A = dg, du or dy by k, B = x or h by k        epilogue: dW
// "by k": stored [k][n], the reduction over rows.  One kernel template covers them: an operand
// stored along k is staged in LDS as [row][64 k]; one stored by k as [64 k][row], read with the
// transposing LDS read.  A product may run over several (A, B) pairs in turn ("segments"): dg and
// du, and the three bf16 terms of an operand carried exactly.
//
// A block owns a BM x BN tile of C; its waves own WM x WN parts of it as 32 x 32 MFMA tiles.
// Both operands stream straight into LDS (16 bytes a lane) into one of two buffers while the
// other is multiplied.
#include <type_traits>

#include "block_internal.h"
#include "common.h"

namespace moe {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

constexpr int kBK = 64;       // reduction indices per step
constexpr int kMaxSeg = 6;
constexpr uint32_t kOob = 0x80000000u;  // an offset past every buffer: reads zero

enum { EPI_STORE = 0, EPI_GU = 1, EPI_DGU = 2 };

struct Seg {
    const uint16_t *a, *b;
};

struct GemmArgs {
    int M, N, K;          // K: reduction length of each segment
    int lda, ldb;         // elements between rows of A and B as stored
    int nseg;
    Seg seg[2][kMaxSeg];  // [blockIdx.y]
    const uint16_t *b2;   // EPI_GU: the up matrix (b of the segment is the gate matrix)
    void *c[2];           // EPI_STORE: [blockIdx.y]
    int ct;
    bool acc;
    // EPI_GU, EPI_DGU
    int act, planes;
    uint16_t *h, *dgu;
    float *gu;            // EPI_GU: written unless null; EPI_DGU: read
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void *p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// One operand's tile of ROWS rows (of the output side) by kBK: its loader and its MFMA fragments.
// KM = false: stored [row][k], LDS [row][64] with the 16-byte chunk c of row r at c ^ (r / 2 % 8).
// KM = true: stored [k][row], LDS [k][ROWS] with chunk c of k at c ^ (4 (k % 4)) (64 rows: 4 (k % 2)):
//   the four k of a transposing read's 16 lanes fall into four 64-byte groups.
// SPAN: the rows of one matrix that the tile covers (half of it where it holds two).
template <int ROWS, bool KM, int NW, int kSpan = ROWS>
struct Tile {
    static constexpr int kSwz = (ROWS / 8 - 1) & 12;
    static constexpr int kInstr = ROWS * kBK * 2 / 1024 / NW;  // 1 KB loads per wave
    static_assert(kInstr >= 1 && kInstr * NW * 1024 == ROWS * kBK * 2, "tile split over the waves");
    uint32_t voff[kInstr];  // byte offset of this lane's piece, without the step's part
    int kc;                 // !KM: first k of the lane's piece
    int rows_left, ld;

    __device__ __forceinline__ void init(int wv, int lane, int rows_left_, int ld_)
    {
        rows_left = rows_left_;
        ld = ld_;
        if constexpr (!KM) {
            // piece i of wave wv: rows 8 (wv kInstr + i) .. + 7
#pragma unroll
            for (int i = 0; i < kInstr; i++) {
                const int r = 8 * (wv * kInstr + i) + (lane >> 3);
                const int c = (lane & 7) ^ ((r >> 1) & 7);
                voff[i] = r < rows_left ? ((uint32_t)r * ld + 8 * c) * 2 : kOob;
            }
        } else {
            constexpr int cpr = ROWS / 8;  // chunks per k
#pragma unroll
            for (int i = 0; i < kInstr; i++) {
                const int s = 64 * (wv * kInstr + i) + lane, k = s / cpr, c = (s % cpr) ^ ((k << 2) & kSwz);
                voff[i] = 8 * c < rows_left ? ((uint32_t)k * ld + 8 * c) * 2 : kOob;
            }
        }
    }

    // Base: the tile's first row at k = 0 of the segment.  rows_left rows (KM: columns) are valid; live =
    // false loads zeros only.  Row offsets of !KM tiles are in voff (the gate/up tile sets its own).
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const uint16_t *base, int k0, int K, bool live) const
    {
        uint32_t bytes;
        if constexpr (!KM) {
            bytes = (uint32_t)(min(rows_left, kSpan) - 1) * ld * 2 + (uint32_t)(K - k0) * 2;
            base += k0;
        } else {
            bytes = (uint32_t)(min(kBK, K - k0) - 1) * ld * 2 + (uint32_t)rows_left * 2;
            base += (size_t)k0 * ld;
        }
        return rsrc_of(base, live ? bytes : 0u);
    }

    // Piece i of the wave; pieces past the reduction's end (a whole number of 16-byte chunks) read zero.
    __device__ __forceinline__ void piece(__amdgpu_buffer_rsrc_t r, uint16_t *lds, int i, int k0, int K, int wv, int lane) const
    {
        uint32_t v = voff[i];
        if constexpr (!KM) {
            const int row = 8 * (wv * kInstr + i) + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
            v = k0 + 8 * c < K ? v : kOob;
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)(lds + 512 * (wv * kInstr + i)), 16,
                                                 (int)v, 0, 0, 0);
    }

    // Fragment of rows row0..row0+31, reduction 16 s..16 s + 15: lane l holds row l % 32, the
    // eight k from 8 (l / 32).
    static __device__ __forceinline__ bf16x8 frag(const uint16_t *lds, int row0, int s, int lane)
    {
        if constexpr (!KM) {
            const int r = row0 + (lane & 31), c = 2 * s + (lane >> 5);
            return as_bf16x8(*(const u32x4 *)(lds + r * kBK + 8 * (c ^ ((r >> 1) & 7))));
        } else {
            // 16-lane group q: rows 16 (q % 2), k from 8 (q / 2); lane i of it addresses k i / 4, rows 4 (i % 4)
            const int q = lane >> 4, i = lane & 15;
            const int k = 16 * s + 8 * (q >> 1) + (i >> 2), row = row0 + 16 * (q & 1) + 4 * (i & 3);
            const uint16_t *p = lds + k * ROWS + ((row & ~7) ^ (((k << 2) & kSwz) << 3)) + (row & 7);
            const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)p);
            const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(p + 4 * ROWS));
            const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
            return as_bf16x8(l2[0], l2[1], h2[0], h2[1]);
        }
    }
};

// Eight consecutive values as `planes` bf16 rows, plane p at dst + p * stride: one rounding, or the
// three terms whose sum is the value (a value that is not finite stays in the first term).
__device__ __forceinline__ void put_planes(uint16_t *dst, size_t stride, int planes, const float (&f)[8])
{
    *(u32x4 *)dst = u32x4{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
    if (planes == 1) return;
    float m[8], l[8];
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const float hi = (float)(__bf16)f[e];
        const bool fin = fabsf(hi) < INFINITY;
        m[e] = fin ? f[e] - hi : 0.f;
        l[e] = m[e] - (float)(__bf16)m[e];
    }
    *(u32x4 *)(dst + stride) = u32x4{bf16_pair(m[0], m[1]), bf16_pair(m[2], m[3]), bf16_pair(m[4], m[5]), bf16_pair(m[6], m[7])};
    *(u32x4 *)(dst + 2 * stride) = u32x4{bf16_pair(l[0], l[1]), bf16_pair(l[2], l[3]), bf16_pair(l[4], l[5]), bf16_pair(l[6], l[7])};
}

__device__ __forceinline__ void put8(float *p, const float (&f)[8])
{
    *(f32x4 *)p = f32x4{f[0], f[1], f[2], f[3]};
    *(f32x4 *)(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
}

// Row r, columns 8 c .. 8 c + 7 of a wave's epilogue scratch.
__device__ __forceinline__ void get8(const f32x4 *sc, int r, int c, float (&f)[8])
{
    const f32x4 a = sc[16 * r + ((2 * c) ^ (r & 15))], b = sc[16 * r + ((2 * c + 1) ^ (r & 15))];
#pragma unroll
    for (int e = 0; e < 4; e++) f[e] = a[e], f[4 + e] = b[e];
}

// Keeps a wave's writes to its own LDS ahead of its other lanes' reads (and the reverse).
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Scheduling hint for the instructions since the last one: the READS LDS reads spread over the MULS
// matrix instructions.
template <int READS, int MULS, int I = 0>
__device__ __forceinline__ void interleave()
{
    constexpr int n = READS < MULS ? READS : MULS;
    if constexpr (I < n) {
        __builtin_amdgcn_sched_group_barrier(0x008, (I + 1) * MULS / n - I * MULS / n, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, (I + 1) * READS / n - I * READS / n, 0);
        interleave<READS, MULS, I + 1>();
    }
}

// The same with LOADS loads into LDS among them.
template <int READS, int LOADS, int MULS, int I = 0>
__device__ __forceinline__ void interleave_loads()
{
    if constexpr (I < MULS) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if constexpr ((I + 1) * LOADS / MULS - I * LOADS / MULS > 0)
            __builtin_amdgcn_sched_group_barrier(0x020, (I + 1) * LOADS / MULS - I * LOADS / MULS, 0);
        if constexpr ((I + 1) * READS / MULS - I * READS / MULS > 0)
            __builtin_amdgcn_sched_group_barrier(0x100, (I + 1) * READS / MULS - I * READS / MULS, 0);
        interleave_loads<READS, LOADS, MULS, I + 1>();
    }
}

// What becomes of eight consecutive values of a product (u: the up values beside gate values v).
template <int EPI>
__device__ __forceinline__ void epilogue(const GemmArgs &g, int z, int m, int n, float (&v)[8], const float (&u)[8])
{
    if constexpr (EPI == EPI_STORE) {
        const size_t at = (size_t)m * g.N + n;
        if (g.ct == DT_F32) {
            float *p = (float *)g.c[z] + at;
            if (g.acc) {
                const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
                for (int e = 0; e < 4; e++) v[e] += a[e], v[4 + e] += b[e];
            }
            put8(p, v);
        } else {
            uint16_t *p = (uint16_t *)g.c[z] + at;
            if (g.acc) {
                const u32x4 b = *(const u32x4 *)p;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    v[2 * e] += __uint_as_float(b[e] << 16);
                    v[2 * e + 1] += __uint_as_float(b[e] & 0xFFFF0000u);
                }
            }
            put_planes(p, 0, 1, v);
        }
    } else if constexpr (EPI == EPI_GU) {
        if (g.h) {
            float h[8];
#pragma unroll
            for (int e = 0; e < 8; e++) h[e] = act_h(g.act, v[e], u[e]);
            put_planes(g.h + (size_t)m * g.N + n, (size_t)g.M * g.N, g.planes, h);
        }
        if (g.gu) {
            float *p = g.gu + (size_t)m * 2 * g.N + n;
            put8(p, v);
            put8(p + g.N, u);
        }
    } else {
        const float *p = g.gu + (size_t)m * 2 * g.N + n;
        float h[8], dg[8], du[8];
#pragma unroll
        for (int q = 0; q < 2; q++) {
            const f32x4 gv = *(const f32x4 *)(p + 4 * q), uv = *(const f32x4 *)(p + g.N + 4 * q);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int k = 4 * q + e;
                act_grad(g.act, gv[e], uv[e], h[k], dg[k], du[k]);
                dg[k] *= v[k];
                du[k] *= v[k];
            }
        }
        if (g.h) put_planes(g.h + (size_t)m * g.N + n, (size_t)g.M * g.N, g.planes, h);
        if (g.dgu) {
            uint16_t *o = g.dgu + (size_t)m * 2 * g.N + n;
            put_planes(o, (size_t)g.M * 2 * g.N, g.planes, dg);
            put_planes(o + g.N, (size_t)g.M * 2 * g.N, g.planes, du);
        }
    }
}

// Tile of the block's index: each XCD (blocks b % 8) takes a run of tiles, walked in groups of
// eight row tiles so that the tiles in flight on one XCD share rows and columns in its L2.
__device__ __forceinline__ void tile_of(int nm, int nn, int &tm, int &tn)
{
    const int n = nm * nn, b = blockIdx.x, x = b & 7, j = b >> 3;
    const int q = n >> 3, rem = n & 7;
    const int t = x * q + min(x, rem) + j;
    constexpr int kGroup = 8;
    const int per = kGroup * nn, g = t / per, m0 = g * kGroup, gm = min(kGroup, nm - m0), r = t - g * per;
    tm = m0 + r % gm;
    tn = r / gm;
}

// WM x WN waves.  EPI_GU: the B tile holds groups of 32 rows, alternately of the gate and the up
// matrix, so a wave's column tiles 2 j and 2 j + 1 are gate and up of the same columns.
template <int BM, int BN, int WM, int WN, bool AK, bool BKM, int EPI>
__global__ __launch_bounds__(64 * WM *WN, 1) void k_ffn_gemm(GemmArgs g)
{
    constexpr int NW = WM * WN, TM = BM / WM / 32, TN = BN / WN / 32;
    constexpr bool GU = EPI == EPI_GU;
    constexpr int BNC = GU ? BN / 2 : BN;  // output columns of a tile
    static_assert(!GU || (TN % 2 == 0 && !BKM), "gate and up tiles pair within a wave");
    __shared__ __attribute__((aligned(1024))) uint16_t as0[BM * kBK], as1[BM * kBK], bs0[BN * kBK], bs1[BN * kBK];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wv / WN, wn = wv % WN;
    int tm, tn;
    tile_of((g.M + BM - 1) / BM, (g.N + BNC - 1) / BNC, tm, tn);
    const int m0 = tm * BM, n0 = tn * BNC, z = blockIdx.y;

    Tile<BM, AK, NW> ta;
    Tile<BN, BKM, NW, BNC> tb;
    ta.init(wv, lane, g.M - m0, g.lda);
    tb.init(wv, lane, g.N - n0, g.ldb);
    if constexpr (GU) {
        // tile row r: matrix r / 32 % 2, output column 32 (r / 64) + r % 32
#pragma unroll
        for (int i = 0; i < tb.kInstr; i++) {
            const int r = 8 * (wv * tb.kInstr + i) + (lane >> 3), col = 32 * (r >> 6) + (r & 31);
            const int c = (lane & 7) ^ ((r >> 1) & 7);
            tb.voff[i] = n0 + col < g.N ? ((uint32_t)col * g.ldb + 8 * c) * 2 : kOob;
        }
    }

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++)
#pragma unroll
            for (int e = 0; e < 16; e++) acc[i][j][e] = 0.f;

    const int ksteps = (g.K + kBK - 1) / kBK, nsteps = ksteps * g.nseg;
    int lseg = 0, lk = 0;  // segment and k of the next load
    // The next tile into as, bs; after the last one zeros, so that the loop needs no branch.
    auto load = [&](uint16_t *as, uint16_t *bs) {
        const bool live = lseg < g.nseg;
        const Seg s = g.seg[z][live ? lseg : 0];
        const auto ra = ta.window(AK ? s.a + m0 : s.a + (size_t)m0 * g.lda, lk, g.K, live);
        const auto rb = tb.window(BKM ? s.b + n0 : s.b + (size_t)n0 * g.ldb, lk, g.K, live);
#pragma unroll
        for (int i = 0; i < ta.kInstr; i++) ta.piece(ra, as, i, lk, g.K, wv, lane);
        if constexpr (GU) {
            const auto ru = tb.window(g.b2 + (size_t)n0 * g.ldb, lk, g.K, live);
#pragma unroll
            for (int i = 0; i < tb.kInstr; i++)  // eight rows, all of one matrix
                tb.piece(((wv * tb.kInstr + i) >> 2) & 1 ? ru : rb, bs, i, lk, g.K, wv, lane);
        } else {
#pragma unroll
            for (int i = 0; i < tb.kInstr; i++) tb.piece(rb, bs, i, lk, g.K, wv, lane);
        }
        lk += kBK;
        const bool over = lk >= g.K;
        lk = over ? 0 : lk;
        lseg += over;
    };
    // Fragments of the 16 reduction indices s of a tile.
    bf16x8 fa[2][TM], fb[2][TN];
    auto read = [&](auto P, const uint16_t *as, const uint16_t *bs, int s) {
        constexpr int p = decltype(P)::value;
#pragma unroll
        for (int j = 0; j < TN; j++) fb[p][j] = Tile<BN, BKM, NW>::frag(bs, 32 * (wn * TN + j), s, lane);
#pragma unroll
        for (int i = 0; i < TM; i++) fa[p][i] = Tile<BM, AK, NW>::frag(as, 32 * (wm * TM + i), s, lane);
    };
    // the B rows (output columns) take the MFMA's row side: a lane ends up with columns
    // 8 q + 4 (lane / 32) + 0..3 of row lane % 32
    auto mul = [&](auto P) {
        constexpr int p = decltype(P)::value;
#pragma unroll
        for (int i = 0; i < TM; i++)
#pragma unroll
            for (int j = 0; j < TN; j++) acc[i][j] = mfma32(fb[p][j], fa[p][i], acc[i][j]);
    };
    using E = std::integral_constant<int, 0>;
    using O = std::integral_constant<int, 1>;
    constexpr int kReads = TN * (BKM ? 2 : 1) + TM * (AK ? 2 : 1), kMul = TM * TN;
    // One tile of 64 k: the fragments of the next 16 k are read while the present ones are multiplied.
    // One barrier a tile, before its last 16 k: by then every wave has read all of this buffer (so the
    // tile after next may stream into it) and has seen its own part of the next tile arrive.
    auto step = [&](const uint16_t *as, const uint16_t *bs, uint16_t *lda_, uint16_t *ldb_, const uint16_t *an, const uint16_t *bn) {
        read(O(), as, bs, 1);
        mul(E());
        interleave<kReads, kMul>();
        read(E(), as, bs, 2);
        mul(O());
        interleave<kReads, kMul>();
        read(O(), as, bs, 3);
        mul(E());
        interleave<kReads, kMul>();
        wait_vm<0>();
        __syncthreads();
        load(lda_, ldb_);
        read(E(), an, bn, 0);  // past the last tile: zeros, not used
        mul(O());
        interleave_loads<kReads, ta.kInstr + tb.kInstr, kMul>();
    };

    load(as0, bs0);
    load(as1, bs1);
    wait_vm<0>();
    __syncthreads();
    read(E(), as0, bs0, 0);
    int st = 0;
    for (; st + 2 <= nsteps; st += 2) {
        step(as0, bs0, as0, bs0, as1, bs1);
        step(as1, bs1, as1, bs1, as0, bs0);
    }
    if (st < nsteps) step(as0, bs0, as0, bs0, as1, bs1);
    wait_vm<0>();  // the zeros behind the last tile have landed before the epilogue uses the buffers
    __syncthreads();

    // Epilogue: a wave's 32 x 64 part at a time goes through its own 8 KB of LDS (16-byte chunk c of a
    // row at c ^ (row % 16)), so that a lane ends up with eight consecutive columns of a row and the
    // stores cover whole lines; the loop over the rows stays rolled.
    uint16_t *const pool[4] = {as0, as1, bs0, bs1};
    constexpr int kPer = NW > 4 ? NW / 4 : 1;
    static_assert(TN % 2 == 0 && kPer * 8192 <= BM * kBK * 2 && kPer * 8192 <= BN * kBK * 2, "epilogue scratch");
    uint16_t *slot = as0;
#pragma unroll
    for (int k = 1; k < 4; k++)
        if (wv / kPer == k) slot = pool[k];
    f32x4 *const sc = (f32x4 *)(slot + 4096 * (wv % kPer));
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j += 2) {
            wave_fence();
#pragma unroll
            for (int d = 0; d < 2; d++)
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const int m = lane & 31, c = 8 * d + 2 * q + (lane >> 5);
                    sc[16 * m + (c ^ (m & 15))] = f32x4{acc[i][j + d][4 * q], acc[i][j + d][4 * q + 1], acc[i][j + d][4 * q + 2], acc[i][j + d][4 * q + 3]};
                }
            wave_fence();
            const int mb = m0 + 32 * (wm * TM + i);
            const int nb = GU ? n0 + 16 * (wn * TN + j) : n0 + 32 * (wn * TN + j);
            constexpr int lpr = GU ? 4 : 8;  // lanes per row
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += 64 / lpr) {
                const int r = r0 + lane / lpr, cb = lane % lpr, m = mb + r, n = nb + 8 * cb;
                float v[8], u[8];
                get8(sc, r, cb, v);
                if constexpr (GU) get8(sc, r, 4 + cb, u);
                if (m < g.M && n < g.N) epilogue<EPI>(g, z, m, n, v, u);
            }
        }
}

template <int BM, int BN, int WM, int WN, bool AK, bool BKM, int EPI>
hipError_t go(const GemmArgs &g, int nz, hipStream_t s)
{
    constexpr int BNC = EPI == EPI_GU ? BN / 2 : BN;
    const size_t tiles = (size_t)((g.M + BM - 1) / BM) * ((g.N + BNC - 1) / BNC);
    hipLaunchKernelGGL((k_ffn_gemm<BM, BN, WM, WN, AK, BKM, EPI>), dim3((unsigned)tiles, (unsigned)nz), dim3(64 * WM * WN), 0, s, g);
    return hipGetLastError();
}

template <bool AK, bool BKM, int EPI>
hipError_t gemm(const GemmArgs &g, int nz, hipStream_t s)
{
    constexpr int cols = EPI == EPI_GU ? 2 : 1;
    const size_t big = (size_t)((g.M + 255) / 256) * ((cols * (size_t)g.N + 255) / 256) * nz;
    if (big >= 200) return go<256, 256, 2, 2, AK, BKM, EPI>(g, nz, s);
    const size_t mid = (size_t)((g.M + 127) / 128) * ((cols * (size_t)g.N + 127) / 128) * nz;
    if (mid >= 200) return go<128, 128, 2, 2, AK, BKM, EPI>(g, nz, s);
    return go<64, 64, 2, 1, AK, BKM, EPI>(g, nz, s);
}

}  // namespace

hipError_t launch_ffn_forward(const FfnArgs &a, hipStream_t s)
{
    const int planes = a.yt == DT_F32 ? kFfnPlanes : 1;
    GemmArgs g{};
    g.M = a.T, g.N = a.I, g.K = a.D, g.lda = g.ldb = a.D, g.nseg = 1;
    g.seg[0][0] = {a.x, a.wg};
    g.b2 = a.wu;
    g.act = a.act, g.planes = planes, g.h = a.h, g.gu = a.gu;
    hipError_t e = gemm<false, false, EPI_GU>(g, 1, s);
    if (e != hipSuccess) return e;
    GemmArgs d{};
    d.M = a.T, d.N = a.D, d.K = a.I, d.lda = d.ldb = a.I, d.nseg = planes;
    for (int p = 0; p < planes; p++) d.seg[0][p] = {a.h + (size_t)p * a.T * a.I, a.wd};
    d.c[0] = a.y, d.ct = a.yt, d.acc = a.acc;
    return gemm<false, false, EPI_STORE>(d, 1, s);
}

hipError_t launch_ffn_backward(const FfnArgs &a, hipStream_t s)
{
    const size_t T = a.T, I = a.I;
    const bool dwgu = a.dwg || a.dwu;
    const int px = a.dx ? (a.dxt == DT_F32 ? kFfnPlanes : 1) : 0;
    const int pw = dwgu || a.dwd ? (a.dwt == DT_F32 ? kFfnPlanes : 1) : 0;
    const float *gu = a.saved_gu;
    hipError_t e;
    if (!gu) {
        GemmArgs g{};
        g.M = a.T, g.N = a.I, g.K = a.D, g.lda = g.ldb = a.D, g.nseg = 1;
        g.seg[0][0] = {a.x, a.wg};
        g.b2 = a.wu;
        g.act = a.act, g.planes = 1, g.gu = a.gu_ws;
        if ((e = gemm<false, false, EPI_GU>(g, 1, s)) != hipSuccess) return e;
        gu = a.gu_ws;
    }
    {
        GemmArgs g{};
        g.M = a.T, g.N = a.I, g.K = a.D, g.lda = a.D, g.ldb = a.I, g.nseg = 1;
        g.seg[0][0] = {a.dy, a.wd};
        g.act = a.act, g.planes = px > pw ? px : pw, g.gu = const_cast<float *>(gu);
        g.h = a.dwd ? a.h : nullptr;
        g.dgu = a.dx || dwgu ? a.dgu : nullptr;
        if ((e = gemm<false, true, EPI_DGU>(g, 1, s)) != hipSuccess) return e;
    }
    if (a.dx) {
        GemmArgs g{};
        g.M = a.T, g.N = a.D, g.K = a.I, g.lda = 2 * a.I, g.ldb = a.D, g.nseg = 2 * px;
        for (int p = 0; p < px; p++) {
            g.seg[0][2 * p] = {a.dgu + p * T * 2 * I, a.wg};
            g.seg[0][2 * p + 1] = {a.dgu + p * T * 2 * I + I, a.wu};
        }
        g.c[0] = a.dx, g.ct = a.dxt, g.acc = a.acc;
        if ((e = gemm<false, true, EPI_STORE>(g, 1, s)) != hipSuccess) return e;
    }
    if (dwgu) {
        GemmArgs g{};
        g.M = a.I, g.N = a.D, g.K = a.T, g.lda = 2 * a.I, g.ldb = a.D, g.nseg = pw;
        int nz = 0;
        for (int m = 0; m < 2; m++) {
            void *out = m ? a.dwu : a.dwg;
            if (!out) continue;
            for (int p = 0; p < pw; p++) g.seg[nz][p] = {a.dgu + p * T * 2 * I + m * I, a.x};
            g.c[nz++] = out;
        }
        g.ct = a.dwt;
        if ((e = gemm<true, true, EPI_STORE>(g, nz, s)) != hipSuccess) return e;
    }
    if (a.dwd) {
        GemmArgs g{};
        g.M = a.D, g.N = a.I, g.K = a.T, g.lda = a.D, g.ldb = a.I, g.nseg = pw;
        for (int p = 0; p < pw; p++) g.seg[0][p] = {a.dy, a.h + p * T * I};
        g.c[0] = a.dwd, g.ct = a.dwt;
        if ((e = gemm<true, true, EPI_STORE>(g, 1, s)) != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace moe
