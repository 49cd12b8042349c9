// ffn.hip -- the dense gated feed-forward block (include/moe_block.h has the formulas).
//
// Five products, all C[m][n] = sum_k A(m, k) B(n, k) in bf16 with fp32 accumulation:
//   gate/up   A = x [T][D],          B = Wg, Wu [I][D]      epilogue: act, h (and g, u)
//   down      A = h [T][I],          B = Wd [D][I]          epilogue: y
//   d h       A = dy [T][D],         B = Wd [D][I] by k     epilogue: act', dg, du, h
//   d x       A = dg | du [T][2I],   B = Wg, Wu [I][D] by k epilogue: dx
//   d W       A = dg, du or dy by k, B = x or h by k        epilogue: dW
// "by k": stored [k][n], the reduction over rows.  One kernel template covers them: an operand
// stored along k is staged in LDS as [row][BK k]; one stored by k as [BK k][row], read with the
// transposing LDS read.  A product may run over several (A, B) pairs in turn ("segments"): dg and
// du, and the three bf16 terms of an operand carried exactly.
//
// A block owns a BM x BN tile of C at a time; its waves own parts of it as 32 x 32 MFMA tiles.  Both
// operands stream straight into LDS (16 bytes a lane) into a ring of four buffers of BK k, three
// steps ahead of the multiplication.  The blocks are persistent: each walks tiles b, b + gridDim, ..., and the stream of
// loads runs on into the next tile while the present one's results are stored through LDS scratch of
// their own, so the matrix pipes wait neither for a first load nor for the last store.
// At 8192 tokens, 7168 -> 14336 -> 7168: gate/up 2.87 ms (1.17 PFLOP/s; 1.28 without keeping g and u), down 1.60
// (1.06), d h 1.70 (0.99), d x 2.72 (1.24), d W 3.78 (1.34); a library's product reaches 1.0 to 1.5 on the card.
// Bound there by how fast 64-byte rows of the tiles arrive in LDS (43 to 58 GB/s a CU) and by the clock that
// the card's power allows (1.8 to 2.0 GHz); d h and gate/up also by the fp32 g and u, whose bytes the epilogue
// moves while no product runs on that CU.  64 k a step in two buffers, whose rows are 128 bytes, cannot ask
// far enough ahead: d W 4.60 ms, d x 2.96.
#include <type_traits>

#include "block_internal.h"
#include "common.h"
#include "ffn_act.h"

namespace moe {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

constexpr int kBufs = 4;      // LDS buffers of a step each
constexpr int kMaxSeg = 6;
constexpr uint32_t kOob = 0x80000000u;  // an offset past every buffer: reads zero

enum { EPI_STORE = 0, EPI_GU = 1, EPI_DGU = 2 };

// One product.
struct Prob {
    int M, N, lda, ldb;  // lda, ldb: elements between rows of A and B as stored
    int tiles;           // number of output tiles (set by the launcher)
    const uint16_t *a[kMaxSeg], *b[kMaxSeg];
    void *c;             // EPI_STORE
    float *part;         // the reduction cut in parts: [splits][M][N], of EPI_GU [splits][M][2N]
};

// Up to three products with the same reduction, walked as one list of tiles.
struct GemmArgs {
    Prob p[3];
    int np, nseg, K;      // K: reduction length of each segment
    int tiles;            // of all products, times splits (set by the launcher, as the next two)
    int splits;           // parts of the reduction, each a tile of its own in the list
    int steps;            // steps of a part, a multiple of kBufs
    int fold;             // > 1: M is this many times the rows of the result, each M / fold rows a term of A; k_ffn_join adds the terms
    const uint16_t *b2;   // EPI_GU: the up matrix (b of the segment is the gate matrix)
    int ct;               // EPI_STORE: dtype of c
    bool acc;
    // EPI_GU, EPI_DGU
    int planes;
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

// One operand's tile of ROWS rows (of the output side) by BK: its loader and its MFMA fragments.
// KM = false: stored [row][k], LDS [row][BK] with the 16-byte chunk c of row r at c ^ (r / 4 % 4) (BK = 64:
//   c ^ (r / 2 % 8)).
// KM = true: stored [k][row], LDS [k][ROWS] with chunk c of k at c ^ (4 (k % 4)) (see swz): the four k of a
//   transposing read's 16 lanes fall into four 64-byte groups.
// Either way no LDS access of a wave meets a bank twice.  SPAN: the rows of one matrix that the tile
// covers (half of it where it holds two).
template <int ROWS, int BK, bool KM, int NW, int SPAN = ROWS>
struct Tile {
    // 256 bytes hold 64 banks: rows of a multiple of them are told apart by two bits of k, 192 rows (384
    // bytes: every second k begins in the other half) and 64 rows by one
    static constexpr int swz(int k) { return ROWS % 128 == 0 ? (k & 3) << 2 : ROWS > 128 ? (k & 2) << 1 : (k & 1) << 2; }
    static constexpr int kInstr = ROWS * BK * 2 / 1024 / NW;  // 1 KB loads per wave
    static constexpr int kCpr = BK / 8, kRpi = 64 / kCpr;     // !KM: chunks of a row, rows of a load
    static constexpr int swz_row(int r) { return BK == 64 ? (r >> 1) & 7 : (r >> 2) & 3; }
    static_assert(kInstr >= 1 && kInstr * NW * 1024 == ROWS * BK * 2, "tile split over the waves");
    static_assert(ROWS % 64 == 0, "a chunk's swizzle stays in its row");
    int chunk[kInstr];      // first k (KM: row) of this lane's piece i
    int line[kInstr];       // its row (KM: k)
    uint32_t voff[kInstr];  // its byte offset in the present product's operand

    __device__ __forceinline__ void init(int wv, int lane)
    {
#pragma unroll
        for (int i = 0; i < kInstr; i++) {
            if constexpr (!KM) {
                line[i] = kRpi * (wv * kInstr + i) + lane / kCpr;
                chunk[i] = 8 * ((lane % kCpr) ^ swz_row(line[i]));
                if (SPAN < ROWS) line[i] = 32 * (line[i] >> 6) + (line[i] & 31);  // groups of 32 rows, alternately of two matrices
            } else {
                constexpr int cpr = ROWS / 8;  // chunks per k
                const int s = 64 * (wv * kInstr + i) + lane;
                line[i] = s / cpr;
                chunk[i] = 8 * ((s % cpr) ^ swz(line[i]));
            }
        }
    }

    // For the tile that the loads turn to: rows of ld elements, of which (KM) left are valid.
    __device__ __forceinline__ void turn(int left, int ld)
    {
#pragma unroll
        for (int i = 0; i < kInstr; i++) {
            voff[i] = ((uint32_t)line[i] * (uint32_t)ld + (uint32_t)chunk[i]) * 2;
            if (KM && chunk[i] >= left) voff[i] = kOob;
        }
    }

    // The part of the operand that a step's pieces may read: base is the tile's first row at k = 0 of the
    // segment, left rows (KM: columns) are valid from there on.  live = false: zeros only.
    static __device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const uint16_t *base, int left, int ld, int k0, int K, bool live)
    {
        uint32_t bytes;
        if constexpr (!KM) {
            // a row past the last begins behind this many bytes, since K - k0 <= ld
            bytes = (uint32_t)(min(left, SPAN) - 1) * ld * 2 + (uint32_t)(K - k0) * 2;
            base += k0;
        } else {
            bytes = (uint32_t)(min(BK, K - k0) - 1) * ld * 2 + (uint32_t)left * 2;
            base += (size_t)k0 * ld;
        }
        return rsrc_of(base, live ? bytes : 0u);
    }

    // Piece i of the wave; of !KM those past the reduction's end (a whole number of 16-byte chunks) read zero.
    __device__ __forceinline__ void piece(__amdgpu_buffer_rsrc_t r, uint16_t *lds, int i, int room, int wv) const
    {
        const uint32_t v = KM || chunk[i] < room ? voff[i] : kOob;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)(lds + 512 * (wv * kInstr + i)), 16,
                                                 (int)v, 0, 0, 0);
    }

    // Fragment of rows row0..row0+31, reduction 16 s..16 s + 15: lane l holds row l % 32, the
    // eight k from 8 (l / 32).
    static __device__ __forceinline__ bf16x8 frag(const uint16_t *lds, int row0, int s, int lane)
    {
        if constexpr (!KM) {
            const int r = row0 + (lane & 31), c = 2 * s + (lane >> 5);
            return as_bf16x8(*(const u32x4 *)(lds + r * BK + 8 * (c ^ swz_row(r))));
        } else {
            // 16-lane group q: rows 16 (q % 2), k from 8 (q / 2); lane i of it addresses k i / 4, rows 4 (i % 4)
            const int q = lane >> 4, i = lane & 15;
            const int k = 16 * s + 8 * (q >> 1) + (i >> 2), row = row0 + 16 * (q & 1) + 4 * (i & 3);
            const uint16_t *p = lds + k * ROWS + ((row & ~7) ^ (swz(k) << 3)) + (row & 7);
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

// A wave's epilogue scratch: one 32 x 32 MFMA tile in fp32, 16-byte chunk c of row r at c ^ (r % 8).
// put_tile takes the accumulator's layout (columns 8 q + 4 (lane / 32) + 0..3 of row lane % 32), get8 a
// row's eight consecutive columns 8 c .. 8 c + 7.
template <typename F>
__device__ __forceinline__ void put_tile(f32x4 *sc, int lane, F &&value)
{
    const int m = lane & 31;
#pragma unroll
    for (int q = 0; q < 4; q++) sc[8 * m + ((2 * q + (lane >> 5)) ^ (m & 7))] = f32x4{value(4 * q), value(4 * q + 1), value(4 * q + 2), value(4 * q + 3)};
}

__device__ __forceinline__ void get8(const f32x4 *sc, int r, int c, float (&f)[8])
{
    const f32x4 a = sc[8 * r + ((2 * c) ^ (r & 7))], b = sc[8 * r + ((2 * c + 1) ^ (r & 7))];
#pragma unroll
    for (int e = 0; e < 4; e++) f[e] = a[e], f[4 + e] = b[e];
}

// f(0), f(1), ... with compile-time numbers, so that what they index stays in registers.
template <int N, typename F, int I = 0>
__device__ __forceinline__ void each(F &&f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        each<N, F, I + 1>(static_cast<F &&>(f));
    }
}

// Keeps a wave's writes to its own LDS ahead of its other lanes' reads (and the reverse).
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_sched_barrier(0);  // and one tile's registers out of the next tile's way
}

// Scheduling hint for the instructions since the last one: an LDS read after each of the first matrix
// instructions, so that the last read has half of them to come back in, and the LOADS loads into LDS
// spread evenly.
template <int READS, int LOADS, int MULS, int I = 0>
__device__ __forceinline__ void interleave()
{
    if constexpr (I < MULS) {
        constexpr int per = (READS + MULS / 2 - 1) / (MULS / 2);  // reads a matrix instruction
        constexpr int reads = I * per < READS ? (READS - I * per < per ? READS - I * per : per) : 0;
        constexpr int loads = (I + 1) * LOADS / MULS - I * LOADS / MULS;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if constexpr (reads > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
        if constexpr (loads > 0) __builtin_amdgcn_sched_group_barrier(0x020, loads, 0);
        interleave<READS, LOADS, MULS, I + 1>();
    }
}

// Eight consecutive values of the product stored, or added onto what is there.
__device__ __forceinline__ void store8(const GemmArgs &g, void *c, size_t at, float (&v)[8])
{
    if (g.ct == DT_F32) {
        float *p = (float *)c + at;
        if (g.acc) {
            const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] += a[e], v[4 + e] += b[e];
        }
        put8(p, v);
    } else {
        uint16_t *p = (uint16_t *)c + at;
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
}

// Eight consecutive gate and up values: kept, and their h.
template <int ACT>
__device__ __forceinline__ void gate8(const GemmArgs &g, int M, int N, int m, int n, const float (&gg)[8], const float (&uu)[8])
{
    if (g.gu) {
        float *p = g.gu + (size_t)m * 2 * N + n;
        put8(p, gg);
        put8(p + N, uu);
    }
    if (g.h) {
        float h[8];
#pragma unroll
        for (int e = 0; e < 8; e++) h[e] = gated<ACT>(gg[e], uu[e]);
        put_planes(g.h + (size_t)m * N + n, (size_t)M * N, g.planes, h);
    }
}

// Eight consecutive values of d h with their saved g and u: h, dg and du.
template <int ACT>
__device__ __forceinline__ void back8(const GemmArgs &g, int M, int N, int m, int n, const float (&dh)[8], const float (&gg)[8],
                                      const float (&uu)[8])
{
    float h[8], dg[8], du[8];
#pragma unroll
    for (int e = 0; e < 8; e++) {
        gated_grad<ACT>(gg[e], uu[e], h[e], dg[e], du[e]);
        dg[e] *= dh[e];
        du[e] *= dh[e];
    }
    if (g.h) put_planes(g.h + (size_t)m * N + n, (size_t)M * N, g.planes, h);
    if (g.dgu) {
        uint16_t *o = g.dgu + (size_t)m * 2 * N + n;
        put_planes(o, (size_t)M * 2 * N, g.planes, dg);
        put_planes(o + N, (size_t)M * 2 * N, g.planes, du);
    }
}

// Place of tile v of the list: its product and first row and column.  Each XCD (v % 8) takes a run of the
// list, walked in groups of eight row tiles so that the tiles in flight on one XCD share rows and
// columns in its L2.
struct Place {
    int p, m0, n0, part;
};

template <int BM, int BNC>
__device__ __forceinline__ Place place_of(const GemmArgs &g, int v)
{
    const int q = g.tiles >> 3, rem = g.tiles & 7, x = v & 7;
    int t = x * q + min(x, rem) + (v >> 3), p = 0;
    const int part = t % g.splits;
    t /= g.splits;
    while (p + 1 < g.np && t >= g.p[p].tiles) t -= g.p[p++].tiles;
    const int nm = (g.p[p].M + BM - 1) / BM, nn = (g.p[p].N + BNC - 1) / BNC;
    constexpr int kGroup = 8;
    const int per = kGroup * nn, grp = t / per, first = grp * kGroup, gm = min(kGroup, nm - first), r = t - grp * per;
    return {p, (first + r % gm) * BM, (r / gm) * BNC, part};
}

// WM x WN waves.  EPI_GU: the B tile holds groups of 32 rows, alternately of the gate and the up
// matrix, so a wave's column tiles 2 j and 2 j + 1 are gate and up of the same columns.
// BK: reduction indices of a step.
template <int BM, int BN, int WM, int WN, int BK, bool AK, bool BKM, int EPI, int ACT>
__global__ __launch_bounds__(64 * WM *WN, 1) void k_ffn_gemm(GemmArgs g)
{
    constexpr int NW = WM * WN, TM = BM / WM / 32, TN = BN / WN / 32;
    constexpr bool GU = EPI == EPI_GU;
    constexpr int BNC = GU ? BN / 2 : BN;  // output columns of a tile
    static_assert(!GU || (TN % 2 == 0 && !BKM), "gate and up tiles pair within a wave");
    // separate arrays, so that the compiler sees that the stream into one does not touch the other
    __shared__ __attribute__((aligned(1024))) uint16_t as0[BM * BK], as1[BM * BK], as2[BM * BK], as3[BM * BK];
    __shared__ __attribute__((aligned(1024))) uint16_t bs0[BN * BK], bs1[BN * BK], bs2[BN * BK], bs3[BN * BK];
    __shared__ f32x4 scratch[NW][256];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wv / WN, wn = wv % WN;

    Tile<BM, BK, AK, NW> ta;
    Tile<BN, BK, BKM, NW, BNC> tb;
    ta.init(wv, lane);
    tb.init(wv, lane);

    f32x16 acc[TM][TN];
    bf16x8 fa[2][TM], fb[2][TN];

    const int ksteps = (g.K + BK - 1) / BK, nsteps = g.steps;  // filled up with steps of zeros
    // The stream of loads: tile, step, segment and k of the next one, and what they read.  All of it is
    // kept in registers: a scalar load in the loop would wait for every LDS read in flight.
    int lv = blockIdx.x, lstep = 0, lseg = 0, lk = 0;
    Place lp;
    const uint16_t *pa, *pb, *pu = nullptr;
    int lda, ldb, lefta, leftb;
    bool live = true;
    auto segment = [&] {
        const Prob &p = g.p[lp.p];
        pa = p.a[lseg] + (AK ? (size_t)lp.m0 : (size_t)lp.m0 * lda);
        pb = p.b[lseg] + (BKM ? (size_t)lp.n0 : (size_t)lp.n0 * ldb);
        if constexpr (GU) pu = g.b2 + (size_t)lp.n0 * ldb;
    };
    auto turn = [&] {
        lp = place_of<BM, BNC>(g, lv);
        const Prob &p = g.p[lp.p];
        lda = p.lda, ldb = p.ldb, lefta = p.M - lp.m0, leftb = p.N - lp.n0;
        ta.turn(lefta, lda);
        tb.turn(leftb, ldb);
        const int first = lp.part * nsteps;
        lseg = first / ksteps;
        lk = (first - lseg * ksteps) * BK;
        live = lseg < g.nseg;
        if (live) segment();
    };
    turn();
    const int K = g.K, nseg = g.nseg, ntiles = g.tiles, nblocks = gridDim.x;
    auto load_a = [&](uint16_t *as) {
        const auto w = ta.window(pa, lefta, lda, lk, K, live);
#pragma unroll
        for (int i = 0; i < ta.kInstr; i++) ta.piece(w, as, i, K - lk, wv);
    };
    auto load_b = [&](uint16_t *bs) {
        const auto w = tb.window(pb, leftb, ldb, lk, K, live);
        if constexpr (GU) {
            const auto wu = tb.window(pu, leftb, ldb, lk, K, live);
#pragma unroll
            for (int i = 0; i < tb.kInstr; i++)  // a load's rows are all of one matrix
                tb.piece((tb.kRpi * (wv * tb.kInstr + i) >> 5) & 1 ? wu : w, bs, i, K - lk, wv);
        } else {
#pragma unroll
            for (int i = 0; i < tb.kInstr; i++) tb.piece(w, bs, i, K - lk, wv);
        }
    };
    auto advance = [&] {
        lk += BK;
        lstep++;
        if (lk < K && lstep < nsteps) return;
        if (lstep == nsteps) {
            lstep = lk = 0;
            lv += nblocks;
            live = lv < ntiles;
            if (live) turn();
        } else {
            lk = 0;
            live = ++lseg < nseg;  // past the last segment: steps of zeros up to the part's length
            if (live) segment();
        }
    };
    // Fragments of the 16 reduction indices s of a tile.
    auto read = [&](auto P, const uint16_t *as, const uint16_t *bs, int s) {
        constexpr int p = decltype(P)::value;
#pragma unroll
        for (int j = 0; j < TN; j++) fb[p][j] = Tile<BN, BK, BKM, NW, BNC>::frag(bs, 32 * (wn * TN + j), s, lane);
#pragma unroll
        for (int i = 0; i < TM; i++) fa[p][i] = Tile<BM, BK, AK, NW>::frag(as, 32 * (wm * TM + i), s, lane);
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
    // One step of BK.  The fragments of the next 16 k are read while the present ones are multiplied, and
    // the loads of the step three further on are spread evenly over the matrix instructions (issued in a
    // bunch they fill the memory pipe's queue, and the wave that waits to issue the next one issues no
    // matrix instruction either).  One barrier a step, before its last 16 k: by then every wave has read
    // all of this buffer (the loads of the next step's turn may stream into it) and has seen its own part
    // of the next step arrive (all but the newest loads: a step's, and what this step has issued).
    constexpr int kSub = BK / 16;
    auto meet = [&] {
        wait_vm<ta.kInstr + tb.kInstr + (kSub > 2 ? ta.kInstr + tb.kInstr : ta.kInstr)>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    auto step = [&](const uint16_t *as, const uint16_t *bs, const uint16_t *an, const uint16_t *bn, uint16_t *al, uint16_t *bl) {
        load_a(al);
        read(O(), as, bs, 1);
        mul(E());
        interleave<kReads, ta.kInstr, kMul>();
        if constexpr (kSub == 4) {
            load_b(bl);
            read(E(), as, bs, 2);
            mul(O());
            interleave<kReads, tb.kInstr, kMul>();
            read(O(), as, bs, 3);
            mul(E());
            interleave<kReads, 0, kMul>();
        }
        meet();
        if constexpr (kSub == 2) load_b(bl);
        read(E(), an, bn, 0);
        mul(O());
        interleave<kReads, kSub == 2 ? tb.kInstr : 0, kMul>();
        advance();
    };

    load_a(as0);
    load_b(bs0);
    advance();
    load_a(as1);
    load_b(bs1);
    advance();
    load_a(as2);
    load_b(bs2);
    advance();
    wait_vm<2 * (ta.kInstr + tb.kInstr)>();
    asm volatile("s_barrier" ::: "memory");
    read(E(), as0, bs0, 0);

    f32x4 *const sc = scratch[wv];
    const int lr = lane >> 2, lc = lane & 3;  // row (of 16) and group of eight columns of the epilogue
    for (int v = blockIdx.x; v < g.tiles; v += gridDim.x) {
        const Place at = place_of<BM, BNC>(g, v);
        const int M = g.p[at.p].M, N = g.p[at.p].N;
        const int mw = at.m0 + 32 * wm * TM, nw = at.n0 + (GU ? 16 : 32) * wn * TN;
#pragma unroll
        for (int i = 0; i < TM; i++)
#pragma unroll
            for (int j = 0; j < TN; j++)
#pragma unroll
                for (int e = 0; e < 16; e++) acc[i][j][e] = 0.f;
        for (int st = 0; st < nsteps; st += kBufs) {
            step(as0, bs0, as1, bs1, as3, bs3);
            step(as1, bs1, as2, bs2, as0, bs0);
            step(as2, bs2, as3, bs3, as1, bs1);
            step(as3, bs3, as0, bs0, as2, bs2);
        }

        // f(row, column, eight values) for each part of the 32 x 32 tile whose value of element e is value(e)
        auto rows = [&](int mb, int nb, auto &&value, auto &&f) {
            wave_fence();
            put_tile(sc, lane, value);
            wave_fence();
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int r = 16 * h + lr;
                float x[8];
                get8(sc, r, lc, x);
                if (mb + r < M && nb + 8 * lc < N) f(h, mb + r, nb + 8 * lc, x);
            }
        };
        if (g.splits > 1 || g.fold > 1) {
            // the part's sums as they are, for k_ffn_join
            const int W = GU ? 2 * N : N;
            float *const part = g.p[at.p].part + (size_t)at.part * M * W;
            each<TM * TN>([&](auto B) {
                constexpr int i = B.value / TN, j = B.value % TN;
                const int nb = GU ? nw + 16 * (j & ~1) : nw + 32 * j;
                rows(mw + 32 * i, nb, [&](int e) { return acc[i][j][e]; },
                     [&](int, int m, int n, float (&x)[8]) { put8(part + (size_t)m * W + (GU && (j & 1) ? N : 0) + n, x); });
            });
            continue;
        }
        if constexpr (EPI == EPI_STORE) {
            void *const c = g.p[at.p].c;
            each<TM * TN>([&](auto B) {
                constexpr int i = B.value / TN, j = B.value % TN;
                rows(mw + 32 * i, nw + 32 * j, [&](int e) { return acc[i][j][e]; },
                     [&](int, int m, int n, float (&x)[8]) { store8(g, c, (size_t)m * N + n, x); });
            });
        } else if constexpr (GU) {
            each<TM * TN / 2>([&](auto B) {
                constexpr int i = B.value / (TN / 2), j = 2 * (B.value % (TN / 2));
                const int mb = mw + 32 * i, nb = nw + 16 * j;
                float gx[2][8];
                rows(mb, nb, [&](int e) { return acc[i][j][e]; },
                     [&](int h, int, int, float (&x)[8]) {
#pragma unroll
                         for (int e = 0; e < 8; e++) gx[h][e] = x[e];
                     });
                rows(mb, nb, [&](int e) { return acc[i][j + 1][e]; },
                     [&](int h, int m, int n, float (&x)[8]) {
                         gate8<ACT>(g, M, N, m, n, gx[h], x);
                     });
            });
        } else {
            // the saved g and u of the next 32 x 32 tile are requested before the present one is worked on
            f32x4 gv[2][2][2], uv[2][2][2];
            auto fetch = [&](auto P, int mb, int nb) {
                constexpr int p = decltype(P)::value;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int m = min(mb + 16 * h + lr, M - 1), n = min(nb + 8 * lc, N - 8);
                    const float *s = g.gu + (size_t)m * 2 * N + n;
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        gv[p][h][q] = *(const f32x4 *)(s + 4 * q);
                        uv[p][h][q] = *(const f32x4 *)(s + N + 4 * q);
                    }
                }
            };
            fetch(E(), mw, nw);
            each<TM * TN>([&](auto B) {
                constexpr int i = B.value / TN, j = B.value % TN, p = B.value & 1, k = B.value + 1;
                if constexpr (k < TM * TN) fetch(std::integral_constant<int, 1 - p>(), mw + 32 * (k / TN), nw + 32 * (k % TN));
                rows(mw + 32 * i, nw + 32 * j, [&](int e) { return acc[i][j][e]; },
                     [&](int h, int m, int n, float (&x)[8]) {
                         float gg[8], uu[8];
#pragma unroll
                         for (int e = 0; e < 8; e++) gg[e] = gv[p][h][e >> 2][e & 3], uu[e] = uv[p][h][e >> 2][e & 3];
                         back8<ACT>(g, M, N, m, n, x, gg, uu);
                     });
            });
        }
    }
}

// Compute units of the current device, down to a multiple of 8 (a grid of such a multiple keeps a block's
// tiles on one XCD).
int compute_units()
{
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess || hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) return 256;
    return n >= 8 ? n & ~7 : 8;
}

// Joins the parts of product blockIdx.y in order, eight columns a thread, and finishes it.
template <int EPI, int ACT>
__global__ __launch_bounds__(256) void k_ffn_join(GemmArgs g)
{
    constexpr bool GU = EPI == EPI_GU;
    const Prob &p = g.p[blockIdx.y];
    const int fold = max(g.fold, 1), M = p.M / fold, N = p.N, terms = g.splits * fold, W = GU ? 2 * N : N, per = N / 8;
    const size_t stride = (size_t)M * W, total = (size_t)M * per;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (size_t)gridDim.x * 256) {
        const int m = (int)(i / per), n = 8 * (int)(i % per);
        const float *src = p.part + (size_t)m * W + n;
        float v[8], u[8];
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] = u[e] = 0.f;
        for (int s = 0; s < terms; s++) {
            const float *q = src + s * stride;
            const f32x4 a = *(const f32x4 *)q, b = *(const f32x4 *)(q + 4);
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] += a[e], v[4 + e] += b[e];
            if constexpr (GU) {
                const f32x4 c = *(const f32x4 *)(q + N), d = *(const f32x4 *)(q + N + 4);
#pragma unroll
                for (int e = 0; e < 4; e++) u[e] += c[e], u[4 + e] += d[e];
            }
        }
        if constexpr (EPI == EPI_STORE) {
            store8(g, p.c, (size_t)m * N + n, v);
        } else if constexpr (GU) {
            gate8<ACT>(g, M, N, m, n, v, u);
        } else {
            const float *q = g.gu + (size_t)m * 2 * N + n;
            float gg[8];
#pragma unroll
            for (int e = 0; e < 8; e++) gg[e] = q[e], u[e] = q[N + e];
            back8<ACT>(g, M, N, m, n, v, gg, u);
        }
    }
}

template <int BM, int BN, int EPI>
int64_t count_tiles(GemmArgs &g)
{
    constexpr int BNC = EPI == EPI_GU ? BN / 2 : BN;
    int64_t n = 0;
    for (int i = 0; i < g.np; i++) {
        const int64_t t = (int64_t)((g.p[i].M + BM - 1) / BM) * ((g.p[i].N + BNC - 1) / BNC);
        g.p[i].tiles = (int)t;
        n += t;
    }
    return n;
}

// slots: blocks that fit the card at once
template <int BM, int BN, int WM, int WN, int BK, bool AK, bool BKM, int EPI, int ACT>
hipError_t go(GemmArgs g, int splits, int slots, hipStream_t s)
{
    const int64_t total = (int64_t)((g.K + BK - 1) / BK) * g.nseg;
    g.steps = (int)(((total + splits - 1) / splits + kBufs - 1) / kBufs * kBufs);
    g.splits = (int)((total + g.steps - 1) / g.steps);
    const int64_t tiles = count_tiles<BM, BN, EPI>(g) * g.splits;
    if (tiles > (int64_t)1 << 30) return hipErrorInvalidValue;
    g.tiles = (int)tiles;
    const unsigned grid = (unsigned)(tiles < slots ? tiles : slots);
    hipLaunchKernelGGL((k_ffn_gemm<BM, BN, WM, WN, BK, AK, BKM, EPI, ACT>), dim3(grid), dim3(64 * WM * WN), 0, s, g);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (g.splits == 1 && g.fold <= 1)) return e;
    size_t most = 0;
    for (int i = 0; i < g.np; i++) most = most > (size_t)g.p[i].M * g.p[i].N ? most : (size_t)g.p[i].M * g.p[i].N;
    if (g.fold > 1) most /= g.fold;
    const size_t blocks = (most / 8 + 255) / 256;
    hipLaunchKernelGGL((k_ffn_join<EPI, ACT>), dim3((unsigned)(blocks < 2048 ? blocks : 2048), (unsigned)g.np), dim3(256), 0, s, g);
    return hipGetLastError();
}

// Microseconds that a product is expected to take with BM x BN tiles and its reduction cut in `splits`.
// From timings of the products at 1 to 8192 tokens, widths 512 to 14336 (the choice takes 1 % more than the
// best tile and cut in the mean, 15 % at most): a step on one CU takes 0.72 us for 256 x 256 tiles of 32 k,
// and 0.47 and 0.23 for 128 x 128 and 64 x 64 tiles of 64 k, so that a large tile does 1.3 and 2.5 times the
// work of the smaller ones in the same time, and wins where it fills the card: 4096 tokens down 147 us
// against 223 and 381, but 1000 tokens d h 73 against 85 and 103, and 400 tokens d h 45 against 38 and 58.
// What comes back from a cut reduction crosses memory twice more in fp32 (6144 -> 3584 at 64 tokens: whole
// 34 us, in four parts 17).  Memory brings what the resident blocks have asked for, three steps each, in 1.2 us.
// The small tiles take 64 k a step because rows of 128 bytes come from memory faster than rows of 64: with
// 32 k, two and four blocks a CU and the same bytes on their way, d x of 400 tokens at 3584 x 6144 took 71 us
// (54 with 64 k), its gate/up 68 (56), down 42 (33); nothing got slower by more than 3 %.
struct Shape {
    int rows, cols, resident, bk;
    double step, cached, alone, tail;  // us per step beside others, per step alone (operands in the last-level cache, in memory), per tile's end
};
constexpr Shape kShapes[4] = {{256, 256, 1, 32, 0.72, 0.54, 0.60, 6.0},
                              {256, 192, 1, 32, 0.64, 0.48, 0.53, 4.5},
                              {128, 128, 1, 64, 0.47, 0.47, 0.49, 0.6},
                              {64, 64, 2, 64, 0.23, 0.28, 0.33, 0.0}};
constexpr double kCached = 32e6;  // operands of fewer bytes are taken to be still cached from the call before

double expected_us(const Shape &c, int64_t tiles, int64_t k, int splits, int fold, int cus, int rows, double in_bytes, double out_bytes,
                   double part_bytes)
{
    const int64_t steps = (k + c.bk - 1) / c.bk;
    const int64_t per = ((steps + splits - 1) / splits + kBufs - 1) / kBufs * kBufs, parts = (steps + per - 1) / per;
    const int64_t blocks = tiles * parts, n = (blocks + cus - 1) / cus;  // n: tiles of the busiest CU
    const double alone = in_bytes < kCached ? c.cached : c.alone, one = c.step * n > alone ? c.step * n : alone;
    double work = per * one + c.tail * n;
    const int64_t resident = blocks < (int64_t)c.resident * cus ? blocks : (int64_t)c.resident * cus;
    const double asked = (double)resident * (kBufs - 1) * c.bk * 2 * (c.cols + (rows < c.rows ? rows : c.rows));
    const double rate = asked / 1.2 < 5.4e6 ? asked / 1.2 : 5.4e6, mem = in_bytes / rate;
    if (mem > work) work = mem;
    return 3.5 + work + out_bytes / 4.4e6 + (parts > 1 || fold > 1 ? 2.1 + 0.4 * parts * fold + 2.0 * parts * part_bytes / 5.6e6 : 0.0);
}

struct Plan {
    int shape = 0, splits = 1;
    double us = 1e30;
};

template <int EPI>
Plan plan(GemmArgs &g, size_t part_floats)
{
    const int cus = compute_units(), fold = g.fold > 1 ? g.fold : 1;
    const int64_t k = (int64_t)g.K * g.nseg;
    size_t floats = 0;
    double in = 0, out = 0;
    int rows = 0;
    for (int i = 0; i < g.np; i++) {
        const Prob &p = g.p[i];
        const double mn = (double)p.M * p.N, wide = EPI == EPI_GU ? 2 : 1;
        floats += (size_t)p.M * p.N * (EPI == EPI_GU ? 2 : 1);
        in += 2.0 * g.K * g.nseg * (p.M + wide * p.N);
        out += EPI == EPI_STORE ? mn / fold * (g.ct == DT_F32 ? 4 : 2)
                                : EPI == EPI_GU ? mn * (2 * (g.h ? g.planes : 0) + (g.gu ? 8 : 0)) : mn * (8 + 2 * g.planes * ((g.h ? 1 : 0) + (g.dgu ? 2 : 0)));
        rows = rows > p.M ? rows : p.M;
    }
    const int64_t tiles[4] = {count_tiles<256, 256, EPI>(g), count_tiles<256, 192, EPI>(g), count_tiles<128, 128, EPI>(g), count_tiles<64, 64, EPI>(g)};
    Plan best;
    for (int c = 0; c < 4; c++)
        for (int sp = 1; sp <= 16 && !(EPI == EPI_GU && c == 1) && ((sp == 1 && fold == 1) || ((sp == 1 || k / sp >= 128) && floats * sp <= part_floats)); sp++) {
            const double t = expected_us(kShapes[c], tiles[c], k, sp, fold, cus, rows, in, out, 4.0 * floats);
            if (t < best.us) best = {c, sp, t};
        }
    return best;
}

template <bool AK, bool BKM, int EPI, int ACT = 0>
hipError_t gemm(GemmArgs g, float *part, size_t part_floats, hipStream_t s)
{
    const int cus = compute_units();
    const Plan c = plan<EPI>(g, part_floats);
    for (int i = 0; i < g.np; i++) {
        g.p[i].part = part;
        part += (size_t)c.splits * g.p[i].M * g.p[i].N * (EPI == EPI_GU ? 2 : 1);
    }
    if (c.shape == 0) return go<256, 256, 2, 2, 32, AK, BKM, EPI, ACT>(g, c.splits, cus, s);
    if constexpr (EPI != EPI_GU)  // gate and up columns pair within a wave: an even number of tiles
        if (c.shape == 1) return go<256, 192, 2, 2, 32, AK, BKM, EPI, ACT>(g, c.splits, cus, s);
    if (c.shape == 2) return go<128, 128, 2, 2, 64, AK, BKM, EPI, ACT>(g, c.splits, cus, s);
    return go<64, 64, 2, 1, 64, AK, BKM, EPI, ACT>(g, c.splits, 2 * cus, s);
}

// The rows of g's one product are terms whose sum is A: g.nseg / terms segments for each of them.  Taken as
// segments, every term reads B again; taken as rows of their own (`fold`), B is read once and the terms'
// sums are joined like parts.  With few tokens B is all there is to read, and the terms' rows fill a tile
// that one term leaves empty: d x of 4 tokens at 6632 x 8008 in fp32 132 -> 60 us, the whole training pass
// of 16 at 3584 x 6144 180 -> 156; with many the rows are tiles of their own, as the segments were, and the
// join is on top.
GemmArgs best_fold(GemmArgs g, int terms, size_t part_floats)
{
    GemmArgs f = g;
    f.fold = terms, f.nseg = g.nseg / terms, f.p[0].M *= terms;
    if (terms > 1 && (int64_t)g.p[0].M * terms < (int64_t)1 << 24 && plan<EPI_STORE>(f, part_floats).us < plan<EPI_STORE>(g, part_floats).us) return f;
    return g;
}

// Product i of g.
Prob &prob(GemmArgs &g, int M, int N, int lda, int ldb, void *c)
{
    Prob &p = g.p[g.np++];
    p.M = M, p.N = N, p.lda = lda, p.ldb = ldb, p.c = c;
    return p;
}

}  // namespace

// What the few-token kernels of ffn_few.hip are expected to take: the weights at 5.6 TB/s, and the tokens,
// which every block reads, from the caches.  At 3584 -> 6144 -> 3584 the two kernels take 18 and 11 us for one
// token (the tiled products 22 and 15) and 46 and 35 for 64 (24 and 17).
static double few_us(int T, int N, int K, int planes, bool pair)
{
    const int tiles = T <= 16 ? 1 : T <= 32 ? 2 : 4, cols = pair ? (tiles == 1 ? 8 : 16) : 16;
    const double weights = 2.0 * (pair ? 2 : 1) * N * K, tokens = (double)((N + cols - 1) / cols) * T * K * 2.0 * planes;
    return 3.0 + weights / 5.6e6 + tokens / (tiles == 1 ? 10e6 : 7e6);
}

// g and u (kept in gu unless null), h in `planes` terms unless null
static hipError_t gate_up(const FfnArgs &a, uint16_t *h, int planes, float *gu, hipStream_t s)
{
    GemmArgs g{};
    Prob &p = prob(g, a.T, a.I, a.D, a.D, nullptr);
    g.nseg = 1, g.K = a.D;
    p.a[0] = a.x, p.b[0] = a.wg, g.b2 = a.wu;
    g.planes = planes, g.h = h, g.gu = gu;
    if (a.T <= kFewTokens && few_us(a.T, a.I, a.D, 1, true) < plan<EPI_GU>(g, a.part_floats).us) return launch_ffn_few_gate_up(a, h, planes, gu, s);
    return a.act == ACT_SITU ? gemm<false, false, EPI_GU, ACT_SITU>(g, a.part, a.part_floats, s)
                             : gemm<false, false, EPI_GU, ACT_SWIGLU>(g, a.part, a.part_floats, s);
}

hipError_t launch_ffn_forward(const FfnArgs &a, hipStream_t s)
{
    const int planes = a.yt == DT_F32 ? kFfnPlanes : 1;
    const hipError_t e = gate_up(a, a.h, planes, a.gu, s);
    if (e != hipSuccess) return e;
    GemmArgs g{};
    Prob &p = prob(g, a.T, a.D, a.I, a.I, a.y);
    g.nseg = planes, g.K = a.I, g.ct = a.yt, g.acc = a.acc;
    for (int k = 0; k < planes; k++) p.a[k] = a.h + (size_t)k * a.T * a.I, p.b[k] = a.wd;
    g = best_fold(g, planes, a.part_floats);
    if (a.T <= kFewTokens && few_us(a.T, a.D, a.I, planes, false) < plan<EPI_STORE>(g, a.part_floats).us) return launch_ffn_few_down(a, planes, s);
    return gemm<false, false, EPI_STORE>(g, a.part, a.part_floats, s);
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
        if ((e = gate_up(a, nullptr, 1, a.gu_ws, s)) != hipSuccess) return e;
        gu = a.gu_ws;
    }
    {
        GemmArgs g{};
        Prob &p = prob(g, a.T, a.I, a.D, a.I, nullptr);
        g.nseg = 1, g.K = a.D;
        p.a[0] = a.dy, p.b[0] = a.wd;
        g.planes = px > pw ? px : pw, g.gu = const_cast<float *>(gu);
        g.h = a.dwd ? a.h : nullptr;
        g.dgu = a.dx || dwgu ? a.dgu : nullptr;
        e = a.act == ACT_SITU ? gemm<false, true, EPI_DGU, ACT_SITU>(g, a.part, a.part_floats, s) : gemm<false, true, EPI_DGU, ACT_SWIGLU>(g, a.part, a.part_floats, s);
        if (e != hipSuccess) return e;
    }
    if (a.dx) {
        GemmArgs g{};
        Prob &p = prob(g, a.T, a.D, 2 * a.I, a.D, a.dx);
        g.nseg = 2 * px, g.K = a.I, g.ct = a.dxt, g.acc = a.acc;
        for (int k = 0; k < px; k++) {
            p.a[2 * k] = a.dgu + k * T * 2 * I, p.b[2 * k] = a.wg;
            p.a[2 * k + 1] = a.dgu + k * T * 2 * I + I, p.b[2 * k + 1] = a.wu;
        }
        g = best_fold(g, px, a.part_floats);
        if ((e = gemm<false, true, EPI_STORE>(g, a.part, a.part_floats, s)) != hipSuccess) return e;
    }
    if (pw) {
        GemmArgs g{};
        g.nseg = pw, g.K = a.T, g.ct = a.dwt;
        for (int m = 0; m < 2; m++) {
            void *out = m ? a.dwu : a.dwg;
            if (!out) continue;
            Prob &p = prob(g, a.I, a.D, 2 * a.I, a.D, out);
            for (int k = 0; k < pw; k++) p.a[k] = a.dgu + k * T * 2 * I + m * I, p.b[k] = a.x;
        }
        if (a.dwd) {
            Prob &p = prob(g, a.D, a.I, a.D, a.I, a.dwd);
            for (int k = 0; k < pw; k++) p.a[k] = a.dy, p.b[k] = a.h + k * T * I;
        }
        return gemm<true, true, EPI_STORE>(g, a.part, a.part_floats, s);
    }
    return hipSuccess;
}

}  // namespace moe
