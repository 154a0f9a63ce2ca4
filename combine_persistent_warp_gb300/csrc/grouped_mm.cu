// grouped_mm.cu -- matrix products with one weight per expert over ragged groups of rows
// (16-bit operands, fp32 accumulators in TMEM).  offsets[e] .. offsets[e+1] are expert e's rows:
//
//   forward   y[r][n]     = sum_k x[r][k] * W[e][n][k]
//   rows      dx[r][k]    = sum_n dy[r][n] * W[e][n][k]
//   weights   dW[e][n][k] = sum_{r of e} dy[r][n] * x[r][k]
//
// Bound by the tensor cores where experts have many rows, by reading the weights where they have
// few.  The 256-wide side of a tile (the UMMA's M, split over a pair of CTAs) is always a
// dimension of the weights: features of the forward product and of the rows' gradient, rows n of
// the weights' gradient.  A ragged group then lies on the UMMA's N, which goes in steps of 32
// rows: a group of m rows is cut into ceil(m/256) tiles whose heights differ by at most one
// step, so a group of any size wastes at most 31 rows, not up to half a 256-row tile, and
// pairs that walk the tile list side by side stay balanced.  In the weights'
// gradient the group is the contracted dimension: each expert has tensor maps of its own that end
// with its last row (a small kernel writes them from the offsets), so TMA fills what a last
// 64-row stage has past the group's end with zeros, in both operands.
//
// Few tiles with a long contraction (small batches, few experts) are split along it: each part
// writes fp32 sums of its own, which a second kernel adds in a fixed order.
//
// Persistent pairs of CTAs (cta_group::2; each CTA holds 128 of the 256 M rows and half of the N
// columns' operand), roles by warp: TMA producer, UMMA issuer (the even CTA's), and the
// epilogue's four warps to each of two TMEM accumulators, drained while the other is filled (the
// weights' gradient, whose shared memory has room for four warps' stores only, has four for both).
// With a short contraction the epilogue bounds: rows' gradient of 42000 x 3320 over 256 in 9 groups 86
// us, 100 with four warps; without one 1% is lost (94 groups of 27 rows, 136 x 88: 9.0 us and 8.9).
// Measured on a GB300, bf16 operands N(0,1) x N(0,0.02): 32 experts of about 1024 rows, N 4096,
// K 7168: forward 1.23-1.31 ms back to back under the power cap (1.47 to 1.56 PFLOP/s; on equal groups
// of 1024 rows 1.18 ms, the library's batched product 1.14 ms), 1.9 PFLOP/s in short bursts, the tensor pipe 86 to
// 90% active; 32 rows an expert: 281 us, 6.8 TB/s of weights; weights' gradient of 128 experts,
// 4096 x 1536, 131072 rows: 1.05-1.10 ms; on equal groups in bursts 0.90 ms, in fp32 1.00, added to an
// fp32 dw 1.26 (its bytes' floor 1.19), added to a 16-bit one 2.28 (add_weights16: a row a lane).  Loads of the shared operand multicast over clusters of four
// CTAs measured the same (144 of 152 SMs in such clusters) and are not used; L2 eviction hints on
// the weights cost up to 6%.
// Operand layouts, both 128-byte swizzled: "K-major" rows of 64 contracted elements, and
// "MN-major" boxes of 64 contracted rows x 64 elements of M or N, so no operand is transposed
// in memory.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "moe_internal.cuh"
#include "op_common.cuh"
#include "ptx.cuh"

using namespace cpw;

namespace {

constexpr int TILE_F = 256;            // M of a pair's UMMA: features of a tile
constexpr int TILE_R = 256;            // N at most: rows (or columns of dW) of a tile
constexpr int KB = 64;                 // contracted elements of a pipeline stage
constexpr int OPER_BYTES = 128 * KB * 2;       // one operand's half in a CTA: 16 KB
constexpr int STAGE = 2 * OPER_BYTES;
constexpr int RING = 6;
template <bool DW>
constexpr int THREADS = DW ? 256 : 384;   // four warps, and four of the epilogue; eight for rows (two tiles at a time)
constexpr int MAX_E = 1024;
constexpr uint64_t WAIT_NS = 2000000000ull;    // limit of every wait but one:
// An accumulator takes as long as its tile has stages, 0.23 us each, and a group of the weights' gradient
// may hold every row there is (2^30 in one of 128 experts: 3.9 s).
constexpr uint64_t STAGE_NS = 2000;
__host__ __device__ constexpr uint64_t tile_wait_ns(int stages) { return WAIT_NS + STAGE_NS * static_cast<uint64_t>(stages); }
static_assert(tile_wait_ns(MAX_ROWS / KB) > 4 * 230 * (MAX_ROWS / KB), "the longest group's products are waited for");
constexpr int STAGE_OUT = 32 * 128;    // dW: an epilogue warp's 32 rows x 128 bytes on their way out
constexpr int ROWS_OUT = 2 * 32 * (256 + 64);   // the other products: 32 rows of two tiles on their way out
constexpr int SMEM = RING * STAGE + 1024 + ROWS_OUT;
constexpr int SMEM_WEIGHTS = RING * STAGE + 1024 + 4 * STAGE_OUT;

__device__ uint32_t g_op_error;        // sticky status of the grouped products (moe_ops_get_error)

// ------------------------------------------------------------------ PTX of CTA pairs ------
__device__ __forceinline__ uint32_t cta_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address in the pair's even CTA of the same shared-memory offset.
__device__ __forceinline__ uint32_t leader_addr(const void *p)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(ptx::smem_u32(p)));
    return a;
}
// Arrivals on a barrier of the even CTA.  They publish no memory, so they are relaxed (a release
// at cluster scope waits for the thread's earlier accesses: 700 cycles a stage on the producer's
// path): TMA orders the operands by its byte counts, and the accumulator's readers have waited
// for their TMEM loads and fenced them.
__device__ __forceinline__ void arrive_relaxed(uint32_t addr)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void arrive_tx_relaxed(uint32_t addr, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(addr), "r"(bytes)
                 : "memory");
}
// Wait for the phase of the given parity, `ns` at most.
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, uint64_t ns = WAIT_NS)
{
    // the timer is read only once a wait has already been long
    uint64_t limit = 0;
    for (uint32_t i = 0;; ++i) {
        if (ptx::mbar_try_wait(bar, parity))
            return true;
        if ((i & 255u) == 255u) {
            const uint64_t now = ptx::globaltimer();
            if (limit == 0)
                limit = now + ns;
            else if (now > limit)
                return false;
        }
    }
}
// Tiled loads into this CTA's shared memory, counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4}], [%2];" ::"r"(ptx::smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void load_3d(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(ptx::smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void umma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}
// The four 16-deep steps of a full stage; A_STEP and B_STEP: a step in descriptor units (16 bytes).
template <int A_STEP, int B_STEP>
__device__ __forceinline__ void umma_pair_stage(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "add.s64 a1, %1, %5;\n\tadd.s64 a2, %1, %6;\n\tadd.s64 a3, %1, %7;\n\t"
                 "add.s64 b1, %2, %8;\n\tadd.s64 b2, %2, %9;\n\tadd.s64 b3, %2, %10;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, 1;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, 1;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(A_STEP), "n"(2 * A_STEP), "n"(3 * A_STEP), "n"(B_STEP),
                 "n"(2 * B_STEP), "n"(3 * B_STEP)
                 : "memory");
}
// Makes a tensor map that a kernel wrote to global memory visible to this thread's TMA loads.
__device__ __forceinline__ void acquire_map(const CUtensorMap *m)
{
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}
// One arrival on the barrier at this offset in both CTAs when the UMMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     ptx::smem_u32(bar)),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
}

// MN-major operand, 128-byte swizzle: boxes of 64 elements of M or N (8 KB apart: leading byte
// offset), 8 contracted rows of 128 bytes each 1024 bytes (stride byte offset).
__device__ __forceinline__ uint64_t mn_major_desc(uint32_t smem_addr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((KB * 128) >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// ------------------------------------------------------------------ the kernel -----------
struct Args {
    int E, F, C;       // experts, features (M side), contracted length (0: ragged rows)
    int R;             // rows of the ragged tensors; dW: columns (N side) of the weights' gradient
    int M;             // rows of the ragged tensors
    const int32_t *offsets;
    void *out;
    long long ldo;     // elements between rows of out
    uint32_t idesc;    // without N
    int f16;           // operands (and a 16-bit out) are fp16, else bf16
    int out32;         // dW: fp32 out
    int accumulate;    // dW: add to out
    const CUtensorMap *maps;   // dW: [E][2] maps of dy and x that end with the expert's rows
    int splits;        // parts of the contraction
    float *part;       // splits > 1: fp32 sums of each part, [splits][M][F] (dW: through map_out)
};

struct Shared {
    uint64_t full[RING], empty[RING];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem;
    int32_t off[MAX_E + 1];     // clamped offsets
    int32_t tile0[MAX_E + 1];   // first tile of each expert
};

enum Kind { FORWARD, ROWS, WEIGHTS };

// Operand geometry of the three products.
template <Kind KIND>
struct Geo {
    static constexpr bool A_MN = KIND != FORWARD;
    static constexpr bool B_MN = KIND == WEIGHTS;
};

// Maps of the K-major operand on the UMMA's N: boxes of 128, 64, 32 and 16 rows.
struct MapsB {
    CUtensorMap m[4];
};

// A tile of the persistent list.
struct Tile {
    int e;         // expert
    int f0;        // first feature
    int r0, rows;  // FORWARD / ROWS: first row and valid rows;  WEIGHTS: first column, valid columns
    int n;         // N of the UMMA (multiple of 32)
    int blocks;    // pipeline stages
    int k0, klen;  // contracted range (WEIGHTS: rows of the group)
    int part;      // of the contraction
};

template <Kind KIND>
struct Tiles {
    const Args &a;
    const Shared &s;
    int total, step, at, e;
    __device__ Tiles(const Args &a_, const Shared &s_) : a(a_), s(s_), e(0)
    {
        total = s.tile0[a.E] * a.splits;   // parts of a tile side by side
        at = blockIdx.x >> 1;
        step = gridDim.x >> 1;
    }
    __device__ bool next(Tile &t)
    {
        if (at >= total)
            return false;
        const int ft = (a.F + TILE_F - 1) / TILE_F;
        const int tile = at / a.splits;
        t.part = at - tile * a.splits;
        if (KIND == WEIGHTS) {
            const int ct = (a.R + TILE_R - 1) / TILE_R;
            t.e = tile / (ft * ct);
            const int i = tile - t.e * (ft * ct);
            t.f0 = (i / ct) * TILE_F;
            t.r0 = (i % ct) * TILE_R;
            t.rows = min(TILE_R, a.R - t.r0);
            t.k0 = s.off[t.e];
            t.klen = s.off[t.e + 1] - t.k0;
        } else {
            while (s.tile0[e + 1] <= tile)
                ++e;
            t.e = e;
            const int m = s.off[e + 1] - s.off[e];
            // the group's units of 32 rows, dealt evenly to its tiles
            const int rt = (m + TILE_R - 1) / TILE_R, units = (m + 31) >> 5;
            const int i = tile - s.tile0[e], r = i % rt;   // rows fastest: the pairs side by side share W
            const int first = r * (units / rt) + min(r, units % rt);
            const int count = units / rt + (r < units % rt ? 1 : 0);
            t.f0 = (i / rt) * TILE_F;
            t.r0 = s.off[e] + 32 * first;
            t.rows = min(32 * count, m - 32 * first);
            t.k0 = 0;
            t.klen = a.C;
        }
        t.n = max(32, (t.rows + 31) & ~31);
        t.blocks = (t.klen + KB - 1) / KB;
        if (a.splits > 1) {
            const int per = (t.blocks + a.splits - 1) / a.splits, before = min(t.blocks, t.part * per);
            t.blocks = min(per, t.blocks - before);
            t.k0 += before * KB;
            t.klen = max(0, min(t.klen - before * KB, per * KB));
        }
        at += step;
        return true;
    }
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int f16)
{
    if (f16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 32 accumulator columns (rows r .. r + 31 of the tile), 128 features f0 .. f0 + 127 of a CTA, one
// feature a lane of the four epilogue warps, into rows of out.  Neighbouring lanes swap halves of
// a pair of rows, so that a lane holds two features of one row; the four warps put their 64 bytes
// of every row into shared memory (rows ROW_PITCH apart: conflict-free) and, behind a barrier, store
// whole 256-byte rows with 16-byte accesses.  (Each warp
// storing its own 64 bytes took 13,600 cycles a tile of 256 rows: 29095 x 2336 x 64 107 us.)
constexpr int ROW_PITCH = 256 + 64;
constexpr int ROW_BUFFER = 32 * ROW_PITCH;
__device__ __forceinline__ void store_rows(const Args &a, const Tile &t, const uint32_t (&v)[32], int r, int f0, int quarter, int lane,
                                           uint8_t *buf, int barrier)
{
    const int odd = lane & 1;
    asm volatile("bar.sync %0, 128;" ::"r"(barrier) : "memory");   // the chunk before has been read
#pragma unroll
    for (int p = 0; p < 16; ++p) {
        const uint32_t own = pack2(__uint_as_float(v[2 * p]), __uint_as_float(v[2 * p + 1]), a.f16);
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
        const uint32_t w = odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
        *reinterpret_cast<uint32_t *>(buf + (2 * p + odd) * ROW_PITCH + quarter * 64 + (lane >> 1) * 4) = w;
    }
    asm volatile("bar.sync %0, 128;" ::"r"(barrier) : "memory");
    uint16_t *out = static_cast<uint16_t *>(a.out);
    const int part = lane & 15, f = f0 + 8 * part;   // 16 lanes a row
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int q = i * 8 + quarter * 2 + (lane >> 4);
        if (r + q < t.rows && f < a.F)
            *reinterpret_cast<uint4 *>(out + static_cast<size_t>(t.r0 + r + q) * a.ldo + f) =
                *reinterpret_cast<const uint4 *>(buf + q * ROW_PITCH + part * 16);
    }
}

// Whether all four epilogue warps have `ok`: they go on, or stop, together.
__device__ __forceinline__ bool epilogue_all(bool ok, int barrier)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(static_cast<uint32_t>(ok)), "r"(barrier)
                 : "memory");
    return r != 0;
}

// 32 accumulator columns of this lane's feature as fp32 sums of a part.
__device__ __forceinline__ void store_part(const Args &a, const Tile &t, const uint32_t (&v)[32], int r, int f)
{
    if (f >= a.F)
        return;
    float *out = a.part + (static_cast<size_t>(t.part) * a.M + t.r0 + r) * a.F + f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (r + i < t.rows)
            out[static_cast<size_t>(i) * a.F] = __uint_as_float(v[i]);
}

// A warp's 32 rows of dW[e] from the accumulator: 128 bytes of each row at a time through the
// warp's shared-memory buffer (swizzled at 128 bytes: conflict-free) and a TMA store, which
// writes whole lines and drops what lies outside [F][R]; in 32 bits the accumulating form is a
// TMA reduction, so the old values are not read by the SM.  (Each lane storing 16 bytes of its
// own row took 12,000 cycles a tile, more than the 8192 of a 1024-row group's products.)
__device__ __forceinline__ void send_weights(const Args &a, const CUtensorMap *map, const Tile &t, const uint8_t *buf, int c, int n0, bool add)
{
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(ptx::smem_u32(buf)), "r"(t.r0 + c), "r"(n0), "r"(t.part * a.E + t.e)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(ptx::smem_u32(buf)), "r"(t.r0 + c), "r"(n0), "r"(t.part * a.E + t.e)
                     : "memory");
    ptx::bulk_commit();
}
template <bool F32>
__device__ __forceinline__ void store_weights(const Args &a, const CUtensorMap *map, const Tile &t, uint32_t src, uint8_t *buf,
                                              int n0, int lane)
{
    constexpr int COLS = F32 ? 32 : 64;   // columns of 128 bytes
    for (int c = 0; c < t.rows; c += COLS) {
        uint32_t w[32];
        if (F32) {
            ptx::tmem_ld32(src + c, w);
            ptx::tmem_ld_wait(w);
        } else {
            uint32_t v[32];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ptx::tmem_ld32(src + c + 32 * h, v);
                ptx::tmem_ld_wait(v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    w[16 * h + i] = pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), a.f16);
            }
        }
        // the previous store has read the buffer
        if (lane == 0)
            ptx::bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4 *>(buf + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0)
            send_weights(a, map, t, buf, c, n0, F32 && a.accumulate);
    }
}
// Zeros for an empty group's rows: one buffer of them feeds all the stores.
__device__ __forceinline__ void store_zeros(const Args &a, const CUtensorMap *map, const Tile &t, uint8_t *buf, int n0, int lane)
{
    if (lane == 0)
        ptx::bulk_wait_read<0>();
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q)
        *reinterpret_cast<uint4 *>(buf + (q * 32 + lane) * 16) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    const int cols = a.out32 ? 32 : 64;
    if (lane == 0)
        for (int c = 0; c < t.rows; c += cols)
            send_weights(a, map, t, buf, c, n0, false);
}

// The accumulating form in 16 bits: 32 columns of this lane's row n, added in fp32 and rounded
// once (a 16-bit TMA reduction would round the product first).
__device__ __forceinline__ void add_weights16(const Args &a, const Tile &t, const uint32_t (&v)[32], int c, int n)
{
    if (n >= a.F)
        return;
    uint16_t *out = static_cast<uint16_t *>(a.out) + (static_cast<size_t>(t.e) * a.F + n) * a.R + t.r0 + c;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (c + 8 * q < t.rows) {
            const uint4 old = *reinterpret_cast<const uint4 *>(out + 8 * q);
            uint32_t w[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 g = a.f16 ? __half22float2(*reinterpret_cast<const __half2 *>(&w[i]))
                                       : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
                w[i] = pack2(__uint_as_float(v[8 * q + 2 * i]) + g.x, __uint_as_float(v[8 * q + 2 * i + 1]) + g.y, a.f16);
            }
            *reinterpret_cast<uint4 *>(out + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

template <Kind KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS<KIND == WEIGHTS>, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ MapsB maps_b,
                   const __grid_constant__ CUtensorMap map_out, const Args a)
{
    extern __shared__ uint8_t raw[];
    __shared__ Shared s;
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();

    if (warp == 0 && lane == 0) {
        if (KIND != WEIGHTS) {
            ptx::prefetch_tmap(&map_a);
            for (int i = 0; i < 4; ++i)
                ptx::prefetch_tmap(&maps_b.m[i]);
        }
    }
    if (warp == 1 && lane == 0) {
        for (int i = 0; i < RING; ++i) {
            ptx::mbar_init(&s.full[i], 2);    // one arrival of each CTA
            ptx::mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&s.acc_full[i], 1);
            ptx::mbar_init(&s.acc_empty[i], 8);   // four epilogue warps of each CTA
        }
        ptx::mbar_init(&s.drain, 1);
        ptx::fence_mbar_init();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(ptx::smem_u32(&s.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    ptx::grid_dependency_wait();   // launched ahead of the end of the kernel before
    if (warp == 3) {
        // offsets clamped to a non-decreasing sequence inside [0, M], whatever they hold, and
        // the number of tiles before each expert
        const int ft = (a.F + TILE_F - 1) / TILE_F;
        int high = 0, tiles = 0;
        for (int e0 = 0; e0 <= a.E; e0 += 32) {
            const int e = e0 + lane;
            int v = e <= a.E ? min(max(a.offsets[e], 0), a.M) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
                if (lane >= o)
                    v = max(v, u);
            }
            v = max(v, high);
            int prev = __shfl_up_sync(0xFFFFFFFFu, v, 1);
            if (lane == 0)
                prev = high;
            // tiles of expert e - 1, which lies between prev and v
            int n = 0;
            if (e >= 1 && e <= a.E)
                n = KIND == WEIGHTS ? ft * ((a.R + TILE_R - 1) / TILE_R) : ft * ((v - prev + TILE_R - 1) / TILE_R);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xFFFFFFFFu, n, o);
                if (lane >= o)
                    n += u;
            }
            n += tiles;
            if (e <= a.E) {
                s.off[e] = v;
                s.tile0[e] = n;
            }
            high = __shfl_sync(0xFFFFFFFFu, v, 31);
            tiles = __shfl_sync(0xFFFFFFFFu, n, 31);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    ptx::tc_fence_after();
    const uint32_t tmem = s.tmem;
    bool ok = true;

    if (warp == 0) {
        // -------------------------------------------------------------------- producer ----
        // (warp-uniform like the issuer: TMA instructions read uniform registers too)
        const uint32_t full0 = __shfl_sync(0xFFFFFFFFu, leader_addr(&s.full[0]), 0);
        const bool issue = elect_one();
        Tiles<KIND> list(a, s);
        Tile t;
        int stage = 0;
        uint32_t phase = 1;
        while (ok && list.next(t)) {
            const int half = t.n >> 1;
            const int fa = t.f0 + static_cast<int>(rank) * 128;
            const int rb = t.r0 + static_cast<int>(rank) * half;
            const int blocks = __shfl_sync(0xFFFFFFFFu, t.blocks, 0);
            // N side: boxes of 64 columns, or the largest box of rows that fits and the smallest
            // one that covers the rest
            int box0 = 0, box1 = 0;
            if (!Geo<KIND>::B_MN) {
                while (box0 < 3 && (128 >> box0) > half)
                    ++box0;
                const int rest = half - (128 >> box0);
                box1 = 3;
                while (rest > (128 >> box1))
                    --box1;
                if (rest <= 0)
                    box1 = -1;
            }
            const int rows_b = Geo<KIND>::B_MN ? (half + 63) / 64 * 64 : (128 >> box0) + (box1 < 0 ? 0 : 128 >> box1);
            const uint32_t bytes = OPER_BYTES + rows_b * 128;
            const int e = t.e;
            // WEIGHTS: the expert's maps (dy, x), written by the kernel before this one
            const CUtensorMap *ea = KIND == WEIGHTS ? a.maps + 2 * e : &map_a, *eb = KIND == WEIGHTS ? ea + 1 : nullptr;
            if (KIND == WEIGHTS && issue) {
                acquire_map(ea);
                acquire_map(eb);
            }
            int k = t.k0;
            for (int b = 0; b < blocks; ++b, k += KB) {
                ok = __all_sync(0xFFFFFFFFu, wait_phase(&s.empty[stage], phase));
                if (!ok)
                    break;
                if (issue) {
                    uint8_t *pa = ring + stage * STAGE, *pb = pa + OPER_BYTES;
                    const uint32_t bar = full0 + stage * 8;
                    arrive_tx_relaxed(bar, bytes);
                    if (KIND == FORWARD) {
                        load_3d(pa, &map_a, bar, k, fa, e);
                    } else if (KIND == ROWS) {
                        load_3d(pa, &map_a, bar, fa, k, e);
                        load_3d(pa + 64 * 128, &map_a, bar, fa + 64, k, e);
                    } else {
                        load_2d(pa, ea, bar, fa, k);
                        load_2d(pa + 64 * 128, ea, bar, fa + 64, k);
                    }
                    if (Geo<KIND>::B_MN) {
                        load_2d(pb, eb, bar, rb, k);
                        if (half > 64)
                            load_2d(pb + 64 * 128, eb, bar, rb + 64, k);
                    } else {
                        load_2d(pb, &maps_b.m[box0], bar, k, rb);
                        if (box1 >= 0)
                            load_2d(pb + (128 >> box0) * 128, &maps_b.m[box1], bar, k, rb + (128 >> box0));
                    }
                }
                __syncwarp();
                if (++stage == RING) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ---------------------------------------------------------------- issuer ------
            // The whole warp runs the loops, one lane issues: with warp-uniform control flow the
            // descriptors stay in uniform registers, which the tcgen05 instructions read (issued
            // from a single lane's branch a stage took 720 to 800 cycles, against the 512 of its
            // products).
            constexpr int A_STEP = Geo<KIND>::A_MN ? 16 * 128 / 16 : 2, B_STEP = Geo<KIND>::B_MN ? 16 * 128 / 16 : 2;
            const uint32_t base = ptx::smem_u32(ring);
            const uint64_t desc_a = Geo<KIND>::A_MN ? mn_major_desc(base) : ptx::kmajor_swizzled_desc<128>(base);
            const uint64_t desc_b = Geo<KIND>::B_MN ? mn_major_desc(base + OPER_BYTES) : ptx::kmajor_swizzled_desc<128>(base + OPER_BYTES);
            const bool issue = elect_one();
            Tiles<KIND> list(a, s);
            Tile t;
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 1;
            while (ok && list.next(t)) {
                const int blocks = __shfl_sync(0xFFFFFFFFu, t.blocks, 0);
                if (blocks == 0)
                    continue;   // an empty group's dW tile: the epilogue writes zeros
                ok = __all_sync(0xFFFFFFFFu, wait_phase(&s.acc_empty[acc], acc_phase));
                if (!ok)
                    break;
                ptx::tc_fence_after();
                const uint32_t d = __shfl_sync(0xFFFFFFFFu, tmem + acc * TILE_R, 0);
                const uint32_t idesc = __shfl_sync(0xFFFFFFFFu, a.idesc | (static_cast<uint32_t>(t.n >> 3) << 17), 0);
                // steps of the last stage (every other one has four)
                const int last = __shfl_sync(0xFFFFFFFFu, (t.klen - (blocks - 1) * KB + 15) / 16, 0);
                for (int b = 0; b < blocks; ++b) {
                    const bool end = b == blocks - 1;
                    ok = __all_sync(0xFFFFFFFFu, wait_phase(&s.full[stage], phase));
                    if (!ok)
                        break;
                    ptx::tc_fence_after();
                    const uint64_t da = desc_a + static_cast<uint32_t>(stage * (STAGE / 16));
                    const uint64_t db = desc_b + static_cast<uint32_t>(stage * (STAGE / 16));
                    if (issue) {
                        if (!end || last == KB / 16) {
                            umma_pair_stage<A_STEP, B_STEP>(d, da, db, idesc, b > 0);
                        } else {
                            for (int i = 0; i < last; ++i)
                                umma_pair(d, da + i * A_STEP, db + i * B_STEP, idesc, b > 0 || i > 0);
                        }
                        commit_pair(&s.empty[stage]);
                        if (end)
                            commit_pair(&s.acc_full[acc]);
                    }
                    __syncwarp();
                    if (++stage == RING) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                acc ^= 1;
                if (acc == 0)
                    acc_phase ^= 1;
            }
            if (!ok) {
                // after a wait that ran out: let the issued UMMAs and the loads in flight land
                if (issue)
                    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                     ptx::smem_u32(&s.drain))
                                 : "memory");
                wait_phase(&s.drain, 0, WAIT_NS / 16);
                for (int i = 0; i < RING; ++i)
                    wait_phase(&s.full[i], i < stage ? phase ^ 1 : phase, WAIT_NS / 16);
            }
        }
    } else if (warp >= 4) {
        // -------------------------------------------------------------------- epilogue ----
        const int quarter = warp & 3, group = (warp >> 2) - 1;
        if (KIND != WEIGHTS && a.splits == 1) {
            // rows that belong to no expert: zero (before the first one only if offsets[0] > 0)
            uint32_t *out = static_cast<uint32_t *>(a.out);
            const int words = a.F / 2;
            const int lo = s.off[0], hi = s.off[a.E];
            for (int i = blockIdx.x; i < lo + a.M - hi; i += gridDim.x) {
                const int row = i < lo ? i : hi + i - lo;
                for (int w = threadIdx.x - 128; w < words; w += blockDim.x - 128)
                    out[(static_cast<size_t>(row) * a.ldo >> 1) + w] = 0;
            }
        }
        Tiles<KIND> list(a, s);
        Tile t;
        int acc = 0;
        uint32_t acc_phase = 0;
        uint8_t *buf = ring + RING * STAGE + quarter * STAGE_OUT;   // WEIGHTS
        while (ok && list.next(t)) {
            const int f0 = t.f0 + static_cast<int>(rank) * 128 + quarter * 32;
            if (KIND == WEIGHTS && t.blocks == 0) {
                if (!a.accumulate && f0 < a.F)
                    store_zeros(a, &map_out, t, buf, f0, lane);
                continue;
            }
            if (KIND != WEIGHTS && acc != group) {   // the other group's accumulator
                acc ^= 1;
                if (acc == 0)
                    acc_phase ^= 1;
                continue;
            }
            ok = __all_sync(0xFFFFFFFFu, wait_phase(&s.acc_full[acc], acc_phase, tile_wait_ns(t.blocks)));
            if (KIND != WEIGHTS)
                ok = epilogue_all(ok, 1 + group);   // store_rows' barriers need all four warps
            if (!ok)
                break;
            ptx::tc_fence_after();
            const uint32_t src = tmem + acc * TILE_R + (static_cast<uint32_t>(quarter * 32) << 16);
            if (KIND == WEIGHTS && (a.out32 || !a.accumulate)) {
                if (f0 < a.F) {
                    if (a.out32)
                        store_weights<true>(a, &map_out, t, src, buf, f0, lane);
                    else
                        store_weights<false>(a, &map_out, t, src, buf, f0, lane);
                }
            } else if (KIND != WEIGHTS && a.splits > 1) {
                // two chunks' registers: a load need not wait for the stores of the chunk before it
                // (850 rows, 5 experts, 128 x 1480: 9.9 us, 13.7 with one)
                uint32_t v[2][32];
                ptx::tmem_ld32(src, v[0]);
                for (int c = 0; c < t.rows; c += 64) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int at = c + 32 * h;
                        if (at >= t.rows)
                            break;
                        ptx::tmem_ld_wait(v[h]);
                        if (at + 32 < t.rows)
                            ptx::tmem_ld32(src + at + 32, v[h ^ 1]);
                        store_part(a, t, v[h], at, f0 + lane);
                    }
                }
            } else {
                for (int c = 0; c < t.rows; c += 32) {
                    uint32_t v[32];
                    ptx::tmem_ld32(src + c, v);
                    ptx::tmem_ld_wait(v);
                    if (KIND == WEIGHTS)
                        add_weights16(a, t, v, c, f0 + lane);
                    else
                        store_rows(a, t, v, c, f0 - quarter * 32, quarter, lane, ring + RING * STAGE + group * ROW_BUFFER, 1 + group);
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0)
                arrive_relaxed(leader_addr(&s.acc_empty[acc]));
            acc ^= 1;
            if (acc == 0)
                acc_phase ^= 1;
        }
        if (KIND == WEIGHTS && lane == 0)
            ptx::bulk_wait<0>();   // the stores read this CTA's shared memory
    }
    if (!ok)
        atomicExch(&g_op_error, static_cast<uint32_t>(MOE_ERR_TIMEOUT));
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// out[r][c] = sum over the parts, in order (+ out if ADD); rows outside [offsets[0], offsets[E]) zero.
struct SumArgs {
    const float *part;
    int splits;
    long long rows, plane;     // plane: rows * width, elements of a part
    int width;
    void *out;
    long long ldo;
    const int32_t *offsets;    // null: every row
    int E, add;
};
template <typename T>
__global__ void __launch_bounds__(256) sum_parts_kernel(const SumArgs a)
{
    ptx::grid_dependency_wait();
    long long lo = 0, hi = a.rows;
    if (a.offsets) {
        // as the products' kernel clamps them: the running maximum, inside [0, rows]
        int top = 0;
        for (int i = threadIdx.x & 31; i <= a.E; i += 32)
            top = max(top, a.offsets[i]);
        hi = min(static_cast<long long>(__reduce_max_sync(0xFFFFFFFFu, top)), a.rows);
        lo = min(static_cast<long long>(max(a.offsets[0], 0)), a.rows);
    }
    const int packs = a.width / 4;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < a.rows * packs; i += gridDim.x * 256ll) {
        const long long row = i / packs;
        const int c = static_cast<int>(i - row * packs) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (row >= lo && row < hi) {
            const float *p = a.part + row * a.width + c;
#pragma unroll 4
            for (int s = 0; s < a.splits; ++s) {
                const float4 q = __ldcs(reinterpret_cast<const float4 *>(p + s * a.plane));
                v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
            }
        }
        T *o = static_cast<T *>(a.out) + row * a.ldo + c;
        if (a.add) {
            v.x += to_f<T>(o[0]), v.y += to_f<T>(o[1]), v.z += to_f<T>(o[2]), v.w += to_f<T>(o[3]);
        }
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4 *>(o) = v;
        } else {
            alignas(8) T h[4] = {from_f<T>(v.x), from_f<T>(v.y), from_f<T>(v.z), from_f<T>(v.w)};
            *reinterpret_cast<uint2 *>(o) = *reinterpret_cast<const uint2 *>(h);
        }
    }
}

// Tensor maps of each expert's rows of dy and x: copies of the whole tensors' maps whose row
// count is the (clamped) end of the expert's group, so that loads past it read zeros.  A warp an
// expert.
constexpr int MAP_WARPS = 4;
__global__ void __launch_bounds__(MAP_WARPS * 32)
    group_maps_kernel(const __grid_constant__ CUtensorMap dy, const __grid_constant__ CUtensorMap x, const int32_t *offsets, int E,
                      int M, CUtensorMap *maps)
{
    ptx::launch_dependents();
    const int e = blockIdx.x * MAP_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (e >= E)
        return;
    int end = 0;
    for (int i = lane; i <= e + 1; i += 32)
        end = max(end, offsets[i]);
    end = min(max(__reduce_max_sync(0xFFFFFFFFu, end), 1), M);   // no stage of an empty group is loaded
    uint32_t *dst = reinterpret_cast<uint32_t *>(maps + 2 * e);
    dst[lane] = reinterpret_cast<const uint32_t *>(&dy)[lane];
    dst[32 + lane] = reinterpret_cast<const uint32_t *>(&x)[lane];
    __syncwarp();
    if (lane < 2) {
        asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(
                         reinterpret_cast<uint64_t>(maps + 2 * e + lane)),
                     "r"(end)
                     : "memory");
        asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
    }
}

// ------------------------------------------------------------------ host side ------------
PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// [d1][d0] (or [d2][d1][d0], slices packed) elements, rows `ld` elements apart, boxes of 128
// bytes x b1 rows, 128-byte swizzle.  Elements outside the tensor read as zero.
bool encode(CUtensorMap *m, const void *base, int dtype, long long d0, long long d1, long long d2, long long ld, int b1)
{
    const cuuint64_t size = dtype_bytes(dtype);
    const auto fn = encoder();
    if (!fn)
        return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1), static_cast<cuuint64_t>(d2)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * size, static_cast<cuuint64_t>(ld) * size * static_cast<cuuint64_t>(d1)};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), static_cast<cuuint32_t>(b1), 1};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(m,
              dtype == MOE_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
              : dtype == MOE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              d2 > 0 ? 3 : 2,
              const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_rows(MapsB &maps, const void *base, int dtype, long long width, long long rows, long long ld)
{
    for (int i = 0; i < 4; ++i)
        if (!encode(&maps.m[i], base, dtype, width, rows, 0, ld, 128 >> i))
            return false;
    return true;
}

// Instruction descriptor of kind::f16 without N: fp32 D, 16-bit A and B, M = 256.
uint32_t instr(bool f16, bool a_mn, bool b_mn)
{
    const uint32_t type = f16 ? 0u : 1u;
    return (1u << 4) | (type << 7) | (type << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(TILE_F >> 4) << 24);
}

template <Kind KIND>
int launch_grouped(const CUtensorMap &ma, const MapsB &mb, const CUtensorMap &mo, const Args &a, int sms, cudaStream_t s)
{
    const auto kern = grouped_kernel<KIND>;
    constexpr int smem = KIND == WEIGHTS ? SMEM_WEIGHTS : SMEM;
    if (ensure_max_dynamic_smem(reinterpret_cast<const void *>(kern), smem) != cudaSuccess)
        return MOE_ERR_CUDA;
    return launch_programmatic(kern, sms / 2 * 2, THREADS<KIND == WEIGHTS>, smem, s, ma, mb, mo, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

bool grouped_sizes_ok(int64_t M, int E, int N, int K, int dtype)
{
    return M >= 0 && M <= MAX_ROWS && E >= 1 && E <= MAX_E && N >= 8 && N % 8 == 0 && K >= 8 && K % 8 == 0 &&
           N <= (1 << 20) && K <= (1 << 20) && (dtype == MOE_BF16 || dtype == MOE_F16);
}

// Parts of the contraction: as many as the idle pairs allow, with at least four stages each, and
// only where the stages saved (0.3 us each) outweigh the second launch (3 us) and the traffic of the
// parts (`out` elements of fp32 each, written and read at 4 TB/s).  Measured, split and not: 16
// rows, one expert, 256 x 7168 9.9 and 25.3 us; 64 rows, 8 experts, 256 x 4096 8.9 and 16.3;
// weights' gradient of 16384 rows, 4 experts, 512 x 512 17.6 and 24.1; 400 rows, 2 experts, 2048 x
// 1024 (not split) 15.1 and 10.1.
int split_count(long long tiles, long long blocks, double out, int sms)
{
    const long long pairs = sms / 2;
    const long long most = tiles > 0 ? (pairs / tiles < blocks / 4 ? pairs / tiles : blocks / 4) : 1;
    int best = 1;
    double gain = 0.0;
    for (long long n = 2; n <= most; ++n) {
        const long long per = (blocks + n - 1) / n, parts = (blocks + per - 1) / per;
        const double g = 0.3 * static_cast<double>(blocks - per) - 3.0 - 8.0 * out * static_cast<double>(parts) / 4e6;
        if (g > gain) {
            gain = g;
            best = static_cast<int>(parts);
        }
    }
    return best;
}
long long div_up(long long a, long long b) { return (a + b - 1) / b; }
int row_splits(int64_t M, int E, int F, int C, int sms)
{
    const long long groups = M < E ? M : E, by_rows = div_up(M, TILE_R);
    return split_count(div_up(F, TILE_F) * (groups > by_rows ? groups : by_rows), div_up(C, KB),
                       static_cast<double>(M) * F, sms);
}
int weight_splits(int64_t M, int E, int N, int K, int sms)
{
    return split_count(E * div_up(N, TILE_F) * div_up(K, TILE_R), div_up(div_up(M, E), KB),
                       static_cast<double>(E) * N * K, sms);
}

template <typename T>
int sum_parts(const SumArgs &a, int sms, cudaStream_t s)
{
    const long long work = a.rows * (a.width / 4), blocks = div_up(work, 256);
    return launch_programmatic(sum_parts_kernel<T>, static_cast<int>(blocks < 8ll * sms ? blocks : 8ll * sms), 256, 0, s, a) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

// Forward product and rows' gradient: F features of out, contraction of length C.
template <Kind KIND>
int run_rows(int64_t M, int E, int F, int C, const CUtensorMap &ma, const MapsB &mb, const int32_t *offsets, void *out, int64_t ldo,
             int dtype, void *workspace, uint64_t workspace_bytes, int sms, cudaStream_t s)
{
    const int splits = row_splits(M, E, F, C, sms);
    const uint64_t need = splits > 1 ? static_cast<uint64_t>(splits) * M * F * sizeof(float) : 0;
    if (need && (!workspace || !op_aligned(workspace, 128) || workspace_bytes < need))
        return MOE_ERR_INVALID_ARG;
    const Args a{E, F, C, 0, static_cast<int>(M), offsets, out, ldo, instr(dtype == MOE_F16, KIND == ROWS, false), dtype == MOE_F16, 0, 0,
                 nullptr, splits, static_cast<float *>(workspace)};
    const int rc = launch_grouped<KIND>(ma, mb, ma, a, sms, s);
    if (rc != MOE_OK || splits == 1)
        return rc;
    const SumArgs q{a.part, splits, M, M * F, F, out, ldo, offsets, E, 0};
    return dtype == MOE_F16 ? sum_parts<__half>(q, sms, s) : sum_parts<__nv_bfloat16>(q, sms, s);
}

bool rows_ok(const void *p, int64_t ld, int width) { return p && op_aligned(p, 16) && ld >= width && ld % 8 == 0; }

}  // namespace

extern "C" {

int moe_grouped_mm_workspace(int64_t M, int E, int N, int K, uint64_t *bytes)
{
    if (!grouped_sizes_ok(M, E, N, K, MOE_BF16) || !bytes)
        return MOE_ERR_INVALID_ARG;
    *bytes = 0;
    if (M == 0)
        return MOE_OK;
    OP_DEVICE(sms);
    // the larger of the forward product's need and the rows' gradient's
    const int fwd = row_splits(M, E, N, K, sms), dx = row_splits(M, E, K, N, sms);
    const uint64_t a = fwd > 1 ? static_cast<uint64_t>(fwd) * M * N : 0, b = dx > 1 ? static_cast<uint64_t>(dx) * M * K : 0;
    *bytes = (a > b ? a : b) * sizeof(float);
    return MOE_OK;
}

int moe_grouped_mm(int64_t M, int E, int N, int K, const void *x, int64_t ldx, const void *w, const int32_t *offsets,
                   void *out, int64_t ldo, int dtype, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (!grouped_sizes_ok(M, E, N, K, dtype))
        return MOE_ERR_INVALID_ARG;
    if (M == 0)
        return MOE_OK;
    if (!rows_ok(x, ldx, K) || !rows_ok(out, ldo, N) || !w || !op_aligned(w, 16) || !offsets || !op_aligned(offsets, 4))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    CUtensorMap ma;
    MapsB mb;
    if (!encode(&ma, w, dtype, K, N, E, K, 128) || !encode_rows(mb, x, dtype, K, M, ldx))
        return MOE_ERR_CUDA;
    return run_rows<FORWARD>(M, E, N, K, ma, mb, offsets, out, ldo, dtype, workspace, workspace_bytes, sms, static_cast<cudaStream_t>(stream));
}

int moe_grouped_mm_dx(int64_t M, int E, int N, int K, const void *dy, int64_t lddy, const void *w, const int32_t *offsets,
                      void *dx, int64_t lddx, int dtype, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (!grouped_sizes_ok(M, E, N, K, dtype))
        return MOE_ERR_INVALID_ARG;
    if (M == 0)
        return MOE_OK;
    if (!rows_ok(dy, lddy, N) || !rows_ok(dx, lddx, K) || !w || !op_aligned(w, 16) || !offsets || !op_aligned(offsets, 4))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    CUtensorMap ma;
    MapsB mb;
    if (!encode(&ma, w, dtype, K, N, E, K, KB) || !encode_rows(mb, dy, dtype, N, M, lddy))
        return MOE_ERR_CUDA;
    return run_rows<ROWS>(M, E, K, N, ma, mb, offsets, dx, lddx, dtype, workspace, workspace_bytes, sms, static_cast<cudaStream_t>(stream));
}

int moe_grouped_mm_dw_workspace(int64_t M, int E, int N, int K, uint64_t *bytes)
{
    if (!grouped_sizes_ok(M, E, N, K, MOE_BF16) || !bytes)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const int splits = weight_splits(M, E, N, K, sms);
    *bytes = 2ull * E * sizeof(CUtensorMap) + (splits > 1 ? static_cast<uint64_t>(splits) * E * N * K * sizeof(float) : 0);
    return MOE_OK;
}

int moe_grouped_mm_dw(int64_t M, int E, int N, int K, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                      const int32_t *offsets, void *dw, int dtype, int dw_dtype, int accumulate, void *workspace,
                      uint64_t workspace_bytes, void *stream)
{
    if (!grouped_sizes_ok(M, E, N, K, dtype) || (dw_dtype != dtype && dw_dtype != MOE_F32) || accumulate < 0 || accumulate > 1)
        return MOE_ERR_INVALID_ARG;
    if (!dw || !op_aligned(dw, 16))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M > 0 && (!rows_ok(dy, lddy, N) || !rows_ok(x, ldx, K) || !offsets || !op_aligned(offsets, 4) ||
                  !workspace || !op_aligned(workspace, 128)))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    uint64_t need = 0;
    if (M > 0 && (moe_grouped_mm_dw_workspace(M, E, N, K, &need) != MOE_OK || workspace_bytes < need))
        return MOE_ERR_INVALID_ARG;
    if (M == 0) {
        if (!accumulate && cudaMemsetAsync(dw, 0, static_cast<size_t>(E) * N * K * dtype_bytes(dw_dtype), s) != cudaSuccess)
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    const int splits = weight_splits(M, E, N, K, sms);
    CUtensorMap *maps = static_cast<CUtensorMap *>(workspace);
    float *part = reinterpret_cast<float *>(maps + 2 * E);
    CUtensorMap mdy, mx, mo;
    if (!encode(&mdy, dy, dtype, N, M, 0, lddy, KB) || !encode(&mx, x, dtype, K, M, 0, ldx, KB) ||
        !(splits > 1 ? encode(&mo, part, MOE_F32, K, N, static_cast<long long>(splits) * E, K, 32)
                     : encode(&mo, dw, dw_dtype, K, N, E, K, 32)))
        return MOE_ERR_CUDA;
    group_maps_kernel<<<(E + MAP_WARPS - 1) / MAP_WARPS, MAP_WARPS * 32, 0, s>>>(mdy, mx, offsets, E, static_cast<int>(M), maps);
    if (launched() != MOE_OK)
        return MOE_ERR_CUDA;
    const Args a{E, N, 0, K, static_cast<int>(M), offsets, dw, K, instr(dtype == MOE_F16, true, true), dtype == MOE_F16,
                 splits > 1 || dw_dtype == MOE_F32, splits > 1 ? 0 : accumulate, maps, splits, part};
    const int rc = launch_grouped<WEIGHTS>(mdy, MapsB{}, mo, a, sms, s);
    if (rc != MOE_OK || splits == 1)
        return rc;
    const long long rows = static_cast<long long>(E) * N;
    const SumArgs q{part, splits, rows, rows * K, K, dw, K, nullptr, E, accumulate};
    return dw_dtype == MOE_F32 ? sum_parts<float>(q, sms, s) : dtype == MOE_F16 ? sum_parts<__half>(q, sms, s) : sum_parts<__nv_bfloat16>(q, sms, s);
}

int moe_ops_get_error(int *device_status, void *stream)
{
    if (!device_status)
        return MOE_ERR_INVALID_ARG;
    *device_status = MOE_OK;
    OP_DEVICE(sms);
    uint32_t v = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyFromSymbolAsync(&v, g_op_error, sizeof(v), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (v) {
        const uint32_t zero = 0;
        if (cudaMemcpyToSymbolAsync(g_op_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
            cudaStreamSynchronize(s) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    *device_status = static_cast<int>(v);
    return MOE_OK;
}

}  // extern "C"
