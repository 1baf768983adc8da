// attn_paged.cuh -- attention of a step's queries over a paged cache of bf16 rows: the whole context, or a sliding
// window and the first tokens.
//
// Query (b, t) at position P = start_pos + t sees the positions p <= P with p > P - window or p < n_first (window 0: all
// p <= P).  Position p is row p % page_size of page table[b, p / page_size]; a row serves as key and value for all heads:
//   s_hp = softmax_scale q_h . k_p,  L_h = ln(sum_p e^{s_hp} + e^{sink_h} + e^{prev_lse_h})
//   out_h = (sum_p e^{s_hp} k_p + e^{prev_lse_h} prev_out_h) / e^{L_h}
//
// The rows that a group's queries see together form its list: the first min(n_first, lo) positions, then lo .. hi (lo:
// the first query's window).  Lists are cut into tiles of 64 rows wherever those lie, so a page may end anywhere in
// a tile and a window of 128 rows is two tiles at any position.  The groups' tiles form one long list that is cut into equal
// contiguous pieces, one per CTA and SM; what a CTA has of a query that others share leaves as an fp32 partial, which a
// second kernel joins.  Where splitting would cost more than it evens out, a list goes to one CTA as a whole.  Two tile buffers; 24 warps:
//   * warps 0..7 run the online softmax (two sets of 32 heads; what P is relative to moves only when a score passes it
//     by 2^8);
//   * warps 8..15 write the outputs, while the next query's tiles are under way: O^T lies in a ring of TMEM blocks;
//   * warps 16..19 copy the rows to the free buffer (16 bytes per thread and copy, past L1 and the registers) as the PV two
//     tiles earlier releases its halves.  Rows that nothing sees are not read but zeros, so that P = 0 meets no NaN;
//   * warp 20 issues the QKs, S^T = tile . Q^T (M = 64 rows, N = heads), warp 21 the PVs, O^T += V^T . P^T (M = 128 dims
//     per block, K = the rows of the tile, the same tile read as an MN-major operand);
//   * warp 22 walks the list, tells the others what comes next and, when decoding, asks for the next tile's rows, into L2;
//   * warp 23 loads Q by TMA as soon as the last QK of the query before has read the buffer.
//
// A long chunk is bound by shared memory: a tile takes 2770 cycles, of which the MMAs read operands in 1790 (counted; at 128 B a
// cycle QK 1024, PV 768) and the other warps' accesses, the rows' copies most of them, take 450; the tensor pipe is active in 1540.
// 2048 queries of 64 heads x 512 at 6144: 2110 us, 0.47 of the measured bf16 peak.  Decoding
// is bound by HBM: 32 queries over 16384 rows 103 us; a tile more costs what its rows take at 6.8 TB/s (81 us for all at the
// measured copy rate), next to 20 us at the start (plan, Q, first tile: 5), the end (parts written 2, joined 4) and between
// the two kernels.  Windows are bound by one query's chain: its Q has to come, the QK of its first tile, the softmax, the
// PV that frees the third tile's buffer; 4096 queries through a window of 128 rows and 4 first ones 181 us, 81 at the
// copy rate.  The code that a query runs through has to stay in the instruction cache: 10 % more of it cost 5 to 9 %.
//
// P is rounded to bf16 for the PV product, as the rows are bf16 and one MMA takes one type: each row's share of the output
// is off by at most 2^-8 of itself, as much as the output's own rounding.  Its sum is taken before, in fp32.
#pragma once
#include <cuda_bf16.h>

#include <atomic>

#include "sti_attn_tiles.cuh"
#include "sti_internal.h"

namespace sti {
namespace {

// ------------------------------------------------------------------ queries and the rows they see

// `pack` consecutive queries of a sequence whose heads together fill the 64 rows of Q (pack = 1: one query).  In memory
// they are one query of pack * h heads.  heads 0: only padding.
struct PagedGroup {
    int b, t0, heads;
    int64_t row0;       // of q, out, prev_out, lse, prev_lse: their first head
};
// A list of rows: row i is position i for i < nf, else lo + (i - nf).
struct PagedRows {
    int nf, lo, n;
};
__device__ __forceinline__ int paged_new(const AttnPagedParams& p, int b) {
    return p.n_new ? min(max(__ldg(p.n_new + b), 0), p.s) : p.s;
}
__device__ __forceinline__ PagedGroup group_of(const AttnPagedParams& p, int u) {
    PagedGroup g;
    g.b = u / p.groups;
    g.t0 = (u - g.b * p.groups) * p.pack;
    g.heads = max(min(p.pack, paged_new(p, g.b) - g.t0), 0) * p.h;
    g.row0 = ((int64_t)g.b * p.s + g.t0) * p.h;
    return g;
}
// first position that the query at position P sees through the window (start_pos < 2^31 and t < 2^30: 32 unsigned bits)
__device__ __forceinline__ uint32_t window_start(const AttnPagedParams& p, uint32_t P) {
    return p.window > 0 && P + 1u > (uint32_t)p.window ? P + 1u - (uint32_t)p.window : 0u;
}
__device__ __forceinline__ PagedRows rows_of(const AttnPagedParams& p, int b, int u) {
    const uint32_t start = (uint32_t)__ldg(p.start_pos + b);
    const int t0 = u * p.pack, t1 = min(t0 + p.pack, paged_new(p, b));
    PagedRows r{0, 0, 0};
    if (t0 >= t1) return r;
    const uint32_t hi = min(start + (uint32_t)t1, (uint32_t)p.cap);   // positions past the table have no row
    r.lo = (int)min(window_start(p, start + (uint32_t)t0), hi);
    r.nf = min(p.n_first, r.lo);
    r.n = r.nf + (int)hi - r.lo;
    return r;
}
__device__ __forceinline__ int group_rows(const AttnPagedParams& p, int b, int u) { return rows_of(p, b, u).n; }

constexpr int kWarps = 24;                     // 8 softmax, 8 output, 4 loading, 4 others
constexpr int kPThreads = 32 * kWarps;
constexpr int kOutWarp = 8, kLoadWarp = 16, kQkWarp = 20, kPvWarp = 21, kListWarp = 22;   // (23 loads Q)
// registers per thread after setmaxnreg: 256 x 104 + 256 x 72 + 128 x 64 + 128 x 64 = 61,440, the 768 x 80 of the launch
constexpr int kRegsSoft = 104, kRegsOut = 72, kRegsLoad = 64, kRegsMma = 64;
constexpr float kTopMost = 8.f;                // log2 of the largest P before its reference moves
constexpr uint32_t kStage = 1024;              // 16 heads x 32 dims of bf16
constexpr uint64_t kRunWaitNs = 1ull << 37;    // 137 s: limit of the waits that last as long as a list, of 2^24 tiles at most (25 s);
                                               // those for a tile have 1 s, and one that runs out ends all
constexpr uint32_t kBarSoft = 3;               // named barriers: 1, 2 the head groups, 3 all softmax warps

// A run of one group's tiles, as the list's warp publishes it.
struct __align__(16) Run {
    int t0, t1;         // tiles t0 .. t1 - 1 of the group's list; t1 = 0: the CTA has no more
    int n, nf;          // rows of the list, and those of them before the window
    int lo, b;          // first position of the window, sequence
    int heads, row0;    // the group's heads, the first one's place among all
    int slot;           // of its partial output, -1: the run holds all of the list
    uint32_t pos;       // position of its first query
    int pad[2];
};
constexpr int kWarpPlan = 256;                 // groups that one warp plans for
constexpr int kRuns = 4, kReaders = 23;        // runs published ahead; the warps that read them

// This CTA's piece of the list of all groups' tiles: tiles lo .. hi - 1, the first one tile `off` of group q's list.
struct Piece {
    long long lo, hi, total;
    int ctas;           // CTAs that have a piece
    int q, off;
};

struct __align__(16) Tail {
    Run run[kRuns];
    float neg_m[2][4][32];    // [head group][warp of the group]: its copy of -reference
    float2 fac[kRuns][64];    // [run % kRuns][head]: the outputs' factors, of O and of prev_out
    float red[2][2][4][32];   // [tile parity][group][warp]: per-warp maxima
    float lsum[2][4][32];
    int vis[2][64];           // [run parity] per head: which rows of the list it sees (kPack), see head_vis
    uint8_t valid[2][8];      // [buffer][row / 8]: bit row % 8: it exists
    int2 start;               // a wide plan's: Piece's q, off
    long long scratch[kWarps];
    // the barriers lie in one row, see init_barriers
    uint64_t full[2][2];      // [buffer][half of the dims] filled
    uint64_t freed[2][2];     // the PV has read it
    uint64_t s_full[2], p_full[2];
    uint64_t q_full[2], q_free[2];                // per half of the dims
    uint64_t o_full[kRuns];                       // a run's PVs are done
    uint64_t fac_full[kRuns];                     // its factors are there
    uint64_t o_free[2][kRuns];                    // the first half of its O, all of it has been read
    uint64_t run_full[kRuns], run_empty[kRuns];
    uint32_t tmem_base;
    int abort;
    int qk_tile;              // tiles whose QK was issued, for the prefetching warp
    int list_done;            // the list's warp publishes no more runs
};

// One barrier per thread.
__device__ __forceinline__ void init_barriers(Tail* tl, int sets) {
    constexpr int kBars = 4 + 4 + 2 + 2 + 4 + 6 * kRuns;
    static_assert(offsetof(Tail, run_empty) + sizeof(tl->run_empty) == offsetof(Tail, full) + kBars * sizeof(uint64_t), "");
    const int i = threadIdx.x;
    if (i >= kBars) return;
    uint32_t count = 1;                                             // freed, s_full, q_full, q_free, o_full, run_full
    if (i < 4) count = (i & 1) == 0 ? 128 + 4 : 128;                // full: every loading thread's copies, in the first half
                                                                    // each warp's `valid` too
    if (i == 10 || i == 11) count = 4 * (uint32_t)sets;             // p_full: the warps that have heads
    if (i >= 16 + kRuns && i < 16 + 2 * kRuns) count = (uint32_t)sets;   // fac_full: a warp of each set
    if (i >= 16 + 2 * kRuns && i < 16 + 4 * kRuns) count = 8;       // o_free: the output warps
    if (i >= kBars - kRuns) count = kReaders;
    mbar_init(&tl->full[0][0] + i, count);
    fence_mbar_init();
}

size_t attn_paged_smem(int d) {
    const int n_cb = (d + 127) / 128 * 2;
    return 1024 + (size_t)n_cb * (kQBlk + 2 * kTBlk) + 2 * kPBuf + 8 * kStage + sizeof(Tail);
}

// Where row i of the run's list lies: its page's number, looked up in the table (-1 past the list), and its place in the page.
struct RowAt {
    int page, row;
};
__device__ __forceinline__ RowAt look_up(const AttnPagedParams& p, const Run& r, int i) {
    if (i >= r.n) return RowAt{-1, 0};
    const uint32_t pos = (uint32_t)(i < r.nf ? i : r.lo + (i - r.nf));
    const uint32_t pg = pos / (uint32_t)p.page_size;
    return RowAt{__ldg(p.table + (int64_t)r.b * p.table_stride + pg), (int)(pos - pg * (uint32_t)p.page_size)};
}
// Its address, null if there is none (past the list; a page outside the pool, which is reported).
__device__ __forceinline__ const uint16_t* row_ptr(const AttnPagedParams& p, const RowAt& at, bool listed) {
    if (at.page < 0 || at.page >= p.n_pages) {
        if (listed && p.status) atomicOr(p.status, 1u /* STI_FLAG_INDEX_RANGE */);
        return nullptr;
    }
    return p.pages + (int64_t)at.page * p.page_stride + (int64_t)at.row * p.d;
}

// Four 8 x 8 matrices of 16-bit values, each turned over on the way: lane 8 i + j gives the address of 8 values that become
// (or were) column j of matrix i, of which lane l has row l / 4, columns 2 (l % 4) and the next.
__device__ __forceinline__ void store_turned(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void load_turned(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Two bf16, an infinity or NaN as -2^-133 (kCleared); cleared: whether there is one such, or there was.  (Both sets of heads look
// at a row, in any order, and have to find the same.)
constexpr uint32_t kCleared = 0x80018001u;
__device__ __forceinline__ uint32_t finite_pair(uint32_t v, bool& cleared) {
    const uint32_t is = __vcmpeq2(v & 0x7F807F80u, 0x7F807F80u);
    cleared = cleared || (is | __vcmpeq2(v, kCleared)) != 0;
    return (v & ~is) | (kCleared & is);
}

// Which rows of the group's list head hd sees: i < n - (v >> 8), and i >= nf + (v & 255) or i < n_first (row i < n_first is
// position i; queries of a group are at most 63 positions apart).
__device__ __forceinline__ int head_vis(const AttnPagedParams& p, const Run& r, int hd) {
    if (hd >= r.heads) return 0x7FFFFF00;   // none of a list that short; what it sees of another goes nowhere
    const uint32_t P = r.pos + (uint32_t)(hd / p.h);
    const uint32_t hi = (uint32_t)(r.lo + (r.n - r.nf));
    const uint32_t end = min(P + 1u, hi);
    const uint32_t lo = min(max(window_start(p, P), (uint32_t)r.lo), hi);
    return (int)((hi - end) << 8 | (lo - (uint32_t)r.lo));
}

// Sum or maximum over the 8 lanes of equal lane % 4 of v[i], in lane 4 j + lane % 4 for i = the bits of j in reverse (7
// exchanges instead of 24).
template <bool MAX>
__device__ __forceinline__ float over_rows(const float (&v)[8]) {
    const int lane = threadIdx.x & 31;
    auto op = [](float x, float y) { return MAX ? fmaxf(x, y) : x + y; };
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float send = lane & 4 ? v[i] : v[i + 4];
        a[i] = op(lane & 4 ? v[i + 4] : v[i], __shfl_xor_sync(kWarpFull, send, 4));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float send = lane & 8 ? a[i] : a[i + 2];
        b[i] = op(lane & 8 ? a[i + 2] : a[i], __shfl_xor_sync(kWarpFull, send, 8));
    }
    const float send = lane & 16 ? b[0] : b[1];
    return op(lane & 16 ? b[1] : b[0], __shfl_xor_sync(kWarpFull, send, 16));
}

// tmem_ld_rows16 of half the heads: g < 2.
__device__ __forceinline__ void tmem_ld_rows16_half(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// Two pieces of 8 dims for a lane, of heads `first` and first + 8 from its own on (zeros past the group's).
__device__ __forceinline__ void load_prev(uint4 (&pre)[2], const uint16_t* at, int first, int there, int d) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        pre[k] = make_uint4(0, 0, 0, 0);
        if (first + 8 * k < there) pre[k] = *reinterpret_cast<const uint4*>(at + (int64_t)(first + 8 * k) * d);
    }
}

// O^T of a warp's 32 heads (TMEM columns at `to`) x 32 dims of a d-block, times the heads' factors in fac (of O, of prev), as
// bf16 to out (kJoins: with prev at the same place; pre: its first pieces, then the next block's if there is one).  Half the heads at a time: a lane has dims l / 4 + 8 i (i < 4) of heads 8 g + 2 (l % 4) + {0, 1}; the 8 x 8 blocks
// are turned over on their way to [16 heads][32 dims] in shared memory at stg, where prev comes from the same way, in
// pieces of 8 dims, two per lane: piece k is head lane / 4 + 8 k, dims 8 (lane % 4) ...  A head's four pieces lie
// turned by (head / 2) % 4, so that neither side meets a bank twice.  out, prev: the lane's first piece; there: heads from
// that one on.  (Turned over in fp32 with scalar stores, a query's outputs took twice as long.)
template <bool kJoins>
__device__ __forceinline__ void write_block(const float2* fac, uint8_t* stg, uint32_t to, uint16_t* out, const uint16_t* prev,
                                            uint4 (&pre)[2], int there, int d, bool another) {
    const int lane = threadIdx.x & 31, l4 = lane & 3, j8 = lane & 7;
    const uint32_t block = smem_u32(stg) + (uint32_t)(j8 * 64 + ((((lane >> 3) + (j8 >> 1)) & 3) << 4));   // + 512 g
    uint4* mine = reinterpret_cast<uint4*>(stg + (lane >> 2) * 64 + (((l4 + (((lane >> 2) & 7) >> 1)) & 3) << 4));
#pragma unroll 1
    for (int h = 0; h < 32; h += 16) {
        uint32_t r[2][8];
        tmem_ld_rows16_half(to + (uint32_t)h, r[0]);
        tmem_ld_rows16_half(to + (uint32_t)h + (16u << 16), r[1]);
        const float4 f[2] = {*reinterpret_cast<const float4*>(fac + h + 2 * l4),
                             *reinterpret_cast<const float4*>(fac + h + 8 + 2 * l4)};   // (of O, of prev) of two heads
        if (kJoins) {
            mine[0] = pre[0];
            mine[32] = pre[1];
            __syncwarp();
            if (h == 0) load_prev(pre, prev, 16, there, d);
            else if (another) load_prev(pre, prev + 128, 0, there, d);
        }
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t w[4], pw[4];
            if (kJoins) load_turned(block + 512u * (uint32_t)g, pw);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x0 = __uint_as_float(r[i >> 1][4 * g + 2 * (i & 1)]) * f[g].x;
                float x1 = __uint_as_float(r[i >> 1][4 * g + 2 * (i & 1) + 1]) * f[g].z;
                if (kJoins) {   // weight 0: prev is not used
                    x0 = f[g].y != 0.f ? x0 + f[g].y * __uint_as_float(pw[i] << 16) : x0;
                    x1 = f[g].w != 0.f ? x1 + f[g].w * __uint_as_float(pw[i] & 0xFFFF0000u) : x1;
                }
                w[i] = pack_bf16x2(x0, x1);
            }
            store_turned(block + 512u * (uint32_t)g, w);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint4 v = mine[32 * k];
            if (h + 8 * k < there) *reinterpret_cast<uint4*>(out + (int64_t)(h + 8 * k) * d) = v;
        }
        __syncwarp();
    }
}

// An MMA that accumulates if acc is not 0, and happens only if `on`.
__device__ __forceinline__ void umma_if(bool on, uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                        uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\t"
        "mov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc), "r"((uint32_t)on)
        : "memory");
}

__device__ __forceinline__ int tiles_of(const AttnPagedParams& p, int q) {
    const int b = q / p.groups;
    return (rows_of(p, b, q - b * p.groups).n + kRows - 1) / kRows;
}

// x / y for quotients and remainders of a list's positions: 64-bit divisions take some hundred cycles, and their code.
__device__ __forceinline__ long long divide(long long x, long long y) {
    return (x | y) >> 32 ? x / y : (long long)((uint32_t)x / (uint32_t)y);
}

// Pieces of total / ctas tiles, the first total % ctas of them one longer; the CTA that has tile x.
__device__ __forceinline__ int piece_of(const Piece& w, long long x) {
    const long long per = divide(w.total, w.ctas), longer = w.total - per * w.ctas;
    return (int)(x < longer * (per + 1) ? divide(x, per + 1) : longer + divide(x - longer * (per + 1), per));
}

// This CTA's piece.  kWide: every thread calls it; else one warp (for few groups: nothing to wait for, and only the warp that
// walks the list has to know; 1 us less).
template <bool kWide>
__device__ __forceinline__ Piece plan_piece(const AttnPagedParams& p, int n, Tail* tl) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = kWide ? threadIdx.x : lane;
    constexpr int kBy = kWide ? kPThreads : 32;
    const int each = n <= kBy ? 1 : (n + kBy - 1) / kBy;
    const long long i0 = (long long)tid * each;
    long long sum = 0;
    for (int k = 0; k < each && i0 + k < n; ++k) sum += tiles_of(p, (int)(i0 + k));
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(kWarpFull, inc, o);
        if (lane >= o) inc += u;
    }
    long long before = 0, total = 0;
    if (kWide) {
        if (lane == 31) tl->scratch[warp] = inc;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const long long u = tl->scratch[k];
            if (k < warp) before += u;
            total += u;
        }
    } else {
        total = __shfl_sync(kWarpFull, inc, 31);
    }
    const long long first = before + inc - sum;
    // as many pieces as make the largest no longer (equal queries are then often cut into equal parts)
    const long long grid = gridDim.x, size = max(divide(total + grid - 1, grid), (long long)p.least);
    const long long pieces = p.whole ? total : divide(total + size - 1, size);
    const int part = (int)blockIdx.x, ctas = pieces < grid ? (int)pieces : (int)grid;
    long long lo = 0, hi = 0;
    if (part < ctas) {
        const long long per = divide(total, ctas), longer = total - per * ctas;
        lo = part * per + (part < longer ? part : longer);
        hi = lo + per + (part < longer ? 1 : 0);
    }
    Piece w{lo, hi, total, ctas, 0, 0};
    bool mine = lo < hi && first <= lo && lo < first + sum;
    if (mine) {
        long long at = first;
        int i = (int)i0;
        if (each > 1)
            for (;; ++i) {
                const int c = tiles_of(p, i);
                if (at + c > lo || i + 1 >= n) break;   // (the second: lengths that another stream changes meanwhile)
                at += c;
            }
        w.q = i;
        w.off = (int)(lo - at);
        if (kWide) tl->start = make_int2(w.q, w.off);
    }
    if (!kWide) {
        const int from = __ffs(__ballot_sync(kWarpFull, mine)) - 1;
        if (from >= 0) {
            w.q = __shfl_sync(kWarpFull, w.q, from);
            w.off = __shfl_sync(kWarpFull, w.off, from);
        }
    }
    return w;
}

// d-blocks of 128 dims; groups of several queries; prev_out to be joined; one group per sequence
template <int NM, bool kPack, bool kJoins, bool kAsks>
__global__ void __launch_bounds__(kPThreads, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const AttnPagedParams p) {
    constexpr int kHalves = (NM + 1) / 2;
    constexpr uint32_t kTile = 2 * NM * kTBlk;
    constexpr uint32_t kTmem = NM == 1 ? 256 : 512;
    // TMEM columns of O^T: d-block m of run r lies in the (r NM + m)-th of a ring of blocks, so that the next run's PVs begin while
    // this one's outputs are written: twice NM blocks, or the six that fit beside S^T (NM = 4: the second half of a run's
    // blocks waits for the first half of the run before).
    constexpr uint32_t kRing = 2 * NM < 6 ? 2 * NM : 6;
    auto o_block = [](uint32_t r, uint32_t m) { return kTmO + 64u * ((r * NM + m) % kRing); };
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int n_cb = p.d / 64;                 // column blocks of 64 dims
    uint8_t* q_s = smem;                       // [2 NM][64 heads][128 B]
    uint8_t* t_s = q_s + 2 * NM * kQBlk;       // two tiles [2 NM][64 rows][128 B]
    uint8_t* p_s = t_s + 2 * kTile;            // two P^T [64 rows][64 heads] bf16
    uint8_t* o_s = p_s + 2 * kPBuf;            // per writing warp: outputs being turned over
    Tail* tl = reinterpret_cast<Tail*>(o_s + 8 * kStage);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nq = p.B * p.groups;
    const int hp = p.pack * p.h;               // heads of a full group
    const int sets = hp > 32 ? 2 : 1;          // sets of 32 heads
    volatile int* abort = &tl->abort;

    init_barriers(tl, sets);
    if (tid == 32) {
        tma_prefetch_desc(&tm_q);
        tl->abort = 0;
        tl->qk_tile = 0;
        tl->list_done = 0;
    }
    if (n_cb & 1)   // the dims past d of the last d-block, which no copy writes
        for (int i = tid; i < 3 * (int)kTBlk / 16; i += kPThreads) {
            const int part = i / (int)(kTBlk / 16), k = i % (int)(kTBlk / 16);   // Q, the tiles (kQBlk = kTBlk)
            reinterpret_cast<uint4*>(q_s + (size_t)(2 * NM * part + n_cb) * kTBlk)[k] = make_uint4(0, 0, 0, 0);
        }
    fence_proxy_async_smem();
    // From here on what earlier kernels wrote is read.  (TMEM after it too: a CTA that held it while it waits could keep it from
    // one of the kernel it waits for.)
    griddep_wait();
    if (warp == kQkWarp) {
        tmem_alloc(&tl->tmem_base, kTmem);
        tmem_relinquish();
    }
    // (a group for each CTA: nothing to plan)
    const bool single = p.whole && nq <= (int)gridDim.x, wide = nq > kWarpPlan;
    Piece piece;
    if (!single && wide) piece = plan_piece<true>(p, nq, tl);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kWarpFull, tl->tmem_base, 0);   // warp-uniform, as the compiler can see
    griddep_launch_dependents();

    // The next run for this warp (false: none, or a wait gave up).  The softmax warps meet at barriers, so they take the same runs
    // whatever waits gave up: all that the list's warp publishes before it ends (which is well before their own limit).
    uint32_t runs = 0;
    auto next_run = [&](Run& r, bool together = false) {
        const uint32_t k = runs % kRuns;
        if (!(together ? warp_wait<true>(&tl->run_full[k], runs / kRuns & 1u, p.status, &tl->list_done, 4 * kRunWaitNs)
                       : warp_wait(&tl->run_full[k], runs / kRuns & 1u, p.status, abort, kRunWaitNs)))
            return false;
        r = tl->run[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(&tl->run_empty[k]);
        ++runs;
        return r.t1 > 0;
    };

    if (warp >= kQkWarp) {
        regs_down<kRegsMma>();
        const int n_mma = (hp + 15) / 16 * 16;
        uint32_t n = 0;
        bool ok = true;   // the whole warp waits, one elected lane issues (so the operands stay warp-uniform)
        auto wait = [&](uint64_t* bar, uint32_t parity, uint64_t limit_ns = STI_WAIT_TIMEOUT_NS) {
            ok = warp_wait(bar, parity, p.status, abort, limit_ns);
            tc_fence_after();
            return ok;
        };
        Run run;
        if (warp == kQkWarp) {
            // -------------------------------------------------------------- QK: the tile and Q, both K-major
            const uint32_t idesc = idesc_bf16_f32(kRows, n_mma, false, false);
            const uint64_t dk = sdesc(smem_u32(t_s), 16, 1024, kLayoutSW128), dq = sdesc(smem_u32(q_s), 16, 1024, kLayoutSW128);
            while (ok && next_run(run)) {
                for (int t = run.t0; t < run.t1 && ok; ++t, ++n) {
                    if (kAsks && lane == 0) tl->qk_tile = (int)n;
                    const uint32_t buf = n & 1u;   // its S^T has been read: the tile was filled after the PV of n - 2
                    // (one half's MMAs as code: with both, what a query runs through no longer fits the instruction cache)
#pragma unroll 1
                    for (int h = 0; h < kHalves; ++h) {
                        if (t == run.t0 && !wait(&tl->q_full[h], (runs - 1) & 1u)) break;
                        if (!wait(&tl->full[buf][h], (n >> 1) & 1u)) break;
                        fence_proxy_async_smem();   // the rows were copied by the loading threads
                        if (elect_one()) {
                            const uint32_t at = opaque(lo32(dk) + buf * (kTile / 16) + (uint32_t)h * (4 * kTBlk / 16));
                            const uint32_t bt = opaque(lo32(dq) + (uint32_t)h * (4 * kQBlk / 16));
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                if (NM % 2 == 0 || k < 8 || 2 * h + 1 < NM)   // (the last half of an odd NM is one d-block)
                                    umma_if(true, tmem + 64u * buf, at + (k >> 2) * (kTBlk / 16) + 2 * (k & 3), hi32(dk),
                                            bt + (k >> 2) * (kQBlk / 16) + 2 * (k & 3), hi32(dq), idesc, h + k);
                            if (t == run.t1 - 1) umma_commit(&tl->q_free[h]);
                            if (h == kHalves - 1) umma_commit(&tl->s_full[buf]);
                        }
                        __syncwarp();
                    }
                }
            }
        } else if (warp == kPvWarp) {
            // -------------------------------------------------------------- PV: the tile and P^T, both MN-major
            const uint32_t idesc = idesc_bf16_f32(128, n_mma, true, true);
            const uint64_t dv = sdesc(smem_u32(t_s), kTBlk, 1024, kLayoutSW128), dp = sdesc(smem_u32(p_s), kPBuf, 1024, kLayoutSW128);
            while (ok && next_run(run)) {
                for (int t = run.t0; t < run.t1; ++t, ++n) {
                    const uint32_t buf = n & 1u;
                    const int steps = (run.n - t * kRows + 15) / 16;   // of 16 rows, four at most
                    if (!wait(&tl->p_full[buf], (n >> 1) & 1u)) break;
                    fence_proxy_async_smem();
                    const uint32_t r = runs - 1;
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        // a run's first tile: its blocks of the ring have been read
                        if (t == run.t0 && h == 0 && r >= 2 && !wait(&tl->o_free[1][(r - 2) % kRuns], (r - 2) / kRuns & 1u)) break;
                        if (t == run.t0 && h == 1 && NM == 4 && r >= 1 && !wait(&tl->o_free[0][(r - 1) % kRuns], (r - 1) / kRuns & 1u))
                            break;
                        if (elect_one()) {
#pragma unroll
                            for (int m = 2 * h; m < NM && m < 2 * h + 2; ++m) {
                                const uint32_t at = opaque(lo32(dv) + buf * (kTile / 16) + (uint32_t)m * (2 * kTBlk / 16));
                                const uint32_t bt = opaque(lo32(dp) + buf * (kPBuf / 16));
                                const uint32_t o = tmem + o_block(r, (uint32_t)m);
#pragma unroll
                                for (int k = 0; k < kRows / 16; ++k)
                                    umma_if(k < steps, o, at + 128 * k, hi32(dv), bt + 128 * k, hi32(dp), idesc,
                                            (uint32_t)(t - run.t0 + k));
                            }
                            umma_commit(&tl->freed[buf][h]);
                            if (h == kHalves - 1 && t == run.t1 - 1) umma_commit(&tl->o_full[r % kRuns]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    __syncwarp();
                }
            }
        } else if (warp == kListWarp) {
            // -------------------------------------------------------------- the runs, and their rows' way to L2
            if (single) {
                piece = Piece{0, 1, 1, 1, (int)blockIdx.x, 0};
            } else if (wide) {
                piece.q = tl->start.x;
                piece.off = tl->start.y;
            } else {
                piece = plan_piece<false>(p, nq, tl);
            }
            long long at_tile = piece.lo;
            int q = piece.q, off = piece.off;
            int2 rec = make_int2(-1, 0);
            while (ok) {
                // the next group with a tile in the piece (p.whole: with its middle there, and then all of it; by their first tiles,
                // 300 queries of 1 to 16 tiles take 60.5 us instead of 55.0, 456 of 13 to 16 109.7 instead of 106.7)
                int nt = 0, u = 0;
                for (; at_tile < piece.hi && q < nq; ++q, off = 0) {   // (the second as in plan_piece)
                    run.b = q / p.groups;
                    u = q - run.b * p.groups;
                    const uint32_t start = (uint32_t)__ldg(p.start_pos + run.b);
                    const int real = paged_new(p, run.b);
                    const PagedRows rows = rows_of(p, run.b, u);
                    run.pos = start + (uint32_t)(u * p.pack);
                    run.heads = max(min(p.pack, real - u * p.pack), 0) * p.h;
                    run.row0 = (run.b * p.s + u * p.pack) * p.h;
                    run.n = rows.n;
                    run.nf = rows.nf;
                    run.lo = rows.lo;
                    nt = (rows.n + kRows - 1) / kRows;
                    const long long mid = at_tile - off + (nt - 1) / 2;
                    if (nt > 0 && (!p.whole || single || (mid >= piece.lo && mid < piece.hi))) break;
                    at_tile += single ? 1 : nt - off;
                    nt = 0;
                }
                const uint32_t k = runs % kRuns;
                if (runs >= kRuns && !wait(&tl->run_empty[k], runs / kRuns - 1 & 1u, kRunWaitNs)) break;
                ++runs;
                run.t0 = run.t1 = 0;
                if (nt > 0) {
                    const long long left = piece.hi - at_tile;
                    run.t0 = p.whole ? 0 : off;
                    run.t1 = p.whole || nt - off < left ? nt : off + (int)left;
                    run.slot = run.t0 == 0 && run.t1 == nt ? -1 : 2 * (int)blockIdx.x + (run.t0 == 0 ? 1 : 0);
                }
                if (lane == 0) {
                    tl->run[k] = run;
                    mbar_arrive(&tl->run_full[k]);
                }
                if (nt == 0) break;
                if (lane == 0) {   // what the run will read first and last
                    const uint32_t bytes = (uint32_t)(run.heads * p.d) * 2u;
                    prefetch_l2_bulk(p.q + (int64_t)run.row0 * p.d, bytes);
                    if (p.prev_out) prefetch_l2_bulk(p.prev_out + (int64_t)run.row0 * p.d, bytes);
                }
                if (run.t0 == 0) {
                    const int last = run.t1 < nt ? piece_of(piece, at_tile + nt - 1) : -1;
                    if (p.by_query && lane == 0) p.rec[q] = make_int2(last < 0 ? -1 : (int)blockIdx.x, last);
                    if (last >= 0) rec = make_int2(q, last);
                }
                at_tile += run.t1 - off;
                ++q;
                off = 0;
                n += (uint32_t)(run.t1 - run.t0);
            }
            __syncwarp();
            if (lane == 0) {
                *static_cast<volatile int*>(&tl->list_done) = 1;
                if (!p.by_query) p.rec[blockIdx.x] = rec;
            }
            // One query group per sequence: of the last runs (a long list's CTA has no more), a tile's rows set out for L2 as soon as
            // the tile before is being copied, for HBM to be kept busy: 32 queries over 16384 rows 102 us, without it 110; two
            // tiles ahead 104, five 117, as what was asked for is dropped from L2 before its turn.  (Several groups find each other's
            // rows in L2, and longer code costs: 4096 queries through a window 143 -> 149 us where it is not even run.)
            if constexpr (kAsks) {
                volatile int* now = &tl->qk_tile;
                __syncwarp();
                const uint32_t last = runs - 1, first = last < kRuns ? 0 : last - (kRuns - 1);   // (the end took a place too)
                for (uint32_t j = first; j < last; ++j) n -= (uint32_t)(tl->run[j % kRuns].t1 - tl->run[j % kRuns].t0);
                for (uint32_t j = first; ok && j < last; ++j) {
                    run = tl->run[j % kRuns];
                    for (int t = run.t0; ok && t < run.t1; ++t, ++n) {
                        for (int i = 0; ok && !__all_sync(kWarpFull, *now + 2 >= (int)n); ++i) {   // (a while at most)
                            ok = __all_sync(kWarpFull, i < 10000000 && !*abort);
                            __nanosleep(100);
                        }
                        // rows that lie side by side in one request each: a warp's bulk prefetches leave it one after another
                        const int i0 = t * kRows + lane;
                        const RowAt l0 = look_up(p, run, i0), l1 = look_up(p, run, i0 + 32);
                        const uint16_t* at[2] = {row_ptr(p, l0, i0 < run.n), row_ptr(p, l1, i0 + 32 < run.n)};
                        unsigned long long a[2], before[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            a[i] = reinterpret_cast<unsigned long long>(at[i]);
                            before[i] = __shfl_up_sync(kWarpFull, a[i], 1);
                        }
                        const unsigned long long mid = __shfl_sync(kWarpFull, a[0], 31);
                        if (lane == 0) {
                            before[0] = 0;
                            before[1] = mid;
                        }
                        const uint32_t bytes = 2u * (uint32_t)p.d;
                        const bool c0 = a[0] && before[0] && a[0] == before[0] + bytes, c1 = a[1] && before[1] && a[1] == before[1] + bytes;
                        const unsigned long long goes_on = (unsigned long long)__ballot_sync(kWarpFull, c1) << 32 | __ballot_sync(kWarpFull, c0);
                        auto length = [&](int i) { return (uint32_t)__ffsll(~((goes_on >> i) >> 1)); };   // of the run of rows from row i on
                        if (a[0] && !c0) prefetch_l2_bulk(at[0], bytes * length(lane));
                        if (a[1] && !c1) prefetch_l2_bulk(at[1], bytes * length(lane + 32));
                    }
                }
            }
        } else {
            // -------------------------------------------------------------- Q
            // Half by half: the first half's buffer is free, and its QK can begin, that much earlier (64 rows of 128 bytes per
            // box, a Q takes some 3000 cycles to come).
            while (ok && next_run(run)) {
                for (int h = 0; h < kHalves && ok; ++h) {
                    if (runs > 1 && !wait(&tl->q_free[h], runs & 1u, kRunWaitNs)) break;
                    // rows past the group's heads are other queries', or zeros past the last: columns of S^T that nothing uses
                    if (elect_one()) {
                        const int cb1 = min(n_cb, 4 * h + 4);
                        mbar_arrive_expect_tx(&tl->q_full[h], (uint32_t)(cb1 - 4 * h) * kQBlk);
                        for (int cb = 4 * h; cb < cb1; ++cb)
                            tma_load_2d(q_s + cb * kQBlk, &tm_q, &tl->q_full[h], 64 * cb, run.row0);
                    }
                    __syncwarp();
                }
            }
        }
        __syncwarp();
    } else if (warp >= kLoadWarp) {
        // -------------------------------------------------------------- tiles
        // The warp's rows are 16 lw .. 16 lw + 15 of each tile; a lane copies 16 bytes of rows 16 lw + lane / 8 + 4 i (i < 4) of
        // every column block, eight lanes a row's 128.
        regs_down<kRegsLoad>();
        const int lw = warp - kLoadWarp, r8 = lane >> 3, ch = lane & 7;
        Run run;
        run.t1 = 0;
        int t = 0;
        bool dead = false;
        // Lane j < 16 looks up where row 16 lw + j lies, a tile ahead of its use: the table's entry takes as long to come as
        // the copies of a tile.
        RowAt ahead{-1, 0};
        bool more = true, listed = false;
        auto next_tile = [&]() {
            if (t == run.t1) {
                more = next_run(run);
                t = run.t0;
                if (!more) return;
            }
            const int i = t * kRows + 16 * lw + (lane & 15);
            listed = i < run.n;
            ahead = look_up(p, run, i);
            ++t;
        };
        next_tile();
        for (uint32_t n = 0; more && !dead; ++n) {
            const uint32_t buf = n & 1u;
            const unsigned long long at = reinterpret_cast<unsigned long long>(row_ptr(p, ahead, listed));
            const uint32_t have = __ballot_sync(kWarpFull, at != 0) & 0xFFFFu;
            const uint16_t* src[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) src[i] = reinterpret_cast<const uint16_t*>(__shfl_sync(kWarpFull, at, r8 + 4 * i));
            next_tile();
            const uint32_t dst = smem_u32(t_s) + buf * kTile + (uint32_t)(16 * lw + r8) * 128u;
#pragma unroll 1
            for (int h = 0; h < kHalves; ++h) {
                if (n >= 2 && !warp_wait(&tl->freed[buf][h], ((n >> 1) - 1) & 1u, p.status, abort)) {
                    dead = true;
                    break;
                }
#pragma unroll
                for (int cb = 0; cb < 4; ++cb) {
                    if (4 * h + cb >= n_cb) break;
#pragma unroll
                    for (int i = 0; i < 4; ++i)   // a row that is not there: zeros, nothing is read
                        cp_async_16(dst + (uint32_t)(4 * h + cb) * kTBlk + 512u * i + (uint32_t)((ch ^ ((r8 + 4 * i) & 7)) << 4),
                                    src[i] ? src[i] + 64 * (4 * h + cb) + 8 * ch : p.out, src[i] ? 16u : 0u);
                }
                cp_async_mbar_arrive_noinc(&tl->full[buf][h]);
                if (h == 0 && lane == 0) {
                    *reinterpret_cast<uint16_t*>(&tl->valid[buf][2 * lw]) = (uint16_t)have;
                    mbar_arrive(&tl->full[buf][0]);
                }
            }
        }
        cp_async_wait<0>();
    } else if (warp >= kOutWarp) {
        // -------------------------------------------------------------- outputs
        // A run's, while the next run's tiles are under way.
        regs_down<kRegsOut>();
        const int lw = warp - kOutWarp, set = lw >> 2, qd = lw & 3;
        const uint32_t lanes = tmem + ((uint32_t)(32 * qd) << 16) + 32u * (uint32_t)set;
        Run run;
        while (next_run(run)) {
            const uint32_t r = runs - 1, k = r % kRuns;
            if (!warp_wait(&tl->fac_full[k], r / kRuns & 1u, p.status, abort, kRunWaitNs)) break;
            if (!warp_wait(&tl->o_full[k], r / kRuns & 1u, p.status, abort)) break;
            tc_fence_after();
            auto read = [&](int half) {   // of O
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tl->o_free[half][k]);
            };
            if (set < sets && run.slot >= 0) {
                // A partial, fp32 [32 dims][4 heads][dim, head]: a lane has a dim, and writes four heads' at a time (128 KB
                // in 2 us; as [head][dim] with 4 bytes per lane and store 5 us).
                const int quads = (hp + 3) / 4;
                float4* po = reinterpret_cast<float4*>(p.part_o) + (int64_t)run.slot * p.d * quads + lane;
#pragma unroll 1
                for (int i = 0; i < 2 * NM; ++i) {
                    if (i == 4) read(0);
                    const int block = 4 * (i >> 1) + qd, quad = 8 * set + 4 * (i & 1);
                    if (32 * block >= p.d) break;
                    uint32_t v[16];
                    tmem_ld16(lanes + o_block(r, (uint32_t)i >> 1) + 16u * (i & 1), v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (quad + j < quads)
                            po[(block * quads + quad + j) * 32] =
                                make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                            __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
                }
            } else if (set < sets) {
                const int64_t first = (int64_t)(run.row0 + 32 * set + (lane >> 2)) * p.d + 32 * qd + 8 * (lane & 3);
                const int there = run.heads - 32 * set - (lane >> 2);
                const uint16_t* prev = (kJoins ? p.prev_out : p.out) + first;
                uint4 pre[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};   // prev of the next step
                if (kJoins) load_prev(pre, prev, 0, there, p.d);
#pragma unroll 1
                for (int m = 0; m < NM; ++m) {
                    if (m == 2) read(0);
                    const int left = p.d - 128 * m - 32 * qd;
                    if (left <= 0) break;
                    write_block<kJoins>(&tl->fac[k][32 * set], o_s + lw * kStage, lanes + o_block(r, (uint32_t)m), p.out + first + 128 * m,
                                prev + 128 * m, pre, there, p.d, left > 128);
                }
            } else if (NM > 2) {
                read(0);
            }
            read(1);
        }
    } else {
        regs_up<kRegsSoft>();
        // -------------------------------------------------------------- softmax
        const int set = warp >> 2, qd = warp & 3;
        const int row = 16 * qd + (lane >> 2);   // this thread's tile rows: row, row + 8
        const int l4 = lane & 3;                 // its heads: 32 set + 8 g + 2 l4 + {0, 1}
        const bool active = set < sets;          // this warp's set has heads
        const uint32_t lane_base = (uint32_t)(32 * qd) << 16;
        const uint32_t bar_set = 1u + (uint32_t)set;
        const float c = p.scale_log2;
        const int own_i = (lane >> 2 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 4);   // over_rows leaves the lane its head own_i,
        const int own_head = 8 * (own_i >> 1) + 2 * l4 + (own_i & 1);                // of the set's 32 this one
        uint32_t n = 0;
        bool dead = false;
        float m_run = -INFINITY;                 // what P is relative to, in log2: lane l: head 32 set + l
        float l_thr[8];                          // running sums of the thread's heads over its rows
        uint32_t saw = 0;                        // bit i: its head i saw a row
        bool unset = true;                       // a head of the set has no reference yet (the same in all of its warps)

        auto mwait = [&](uint64_t* bar, uint32_t parity) {
            if (!dead) dead = !warp_wait(bar, parity, p.status, abort);
        };

        // One tile's probabilities 2^(S c - m), m the head's reference.
        float nm[8];
        auto load_m = [&]() {   // from the warp's copy, which has every head of the group
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float2 v = *reinterpret_cast<const float2*>(&tl->neg_m[set][qd][8 * g + 2 * l4]);
                nm[2 * g] = v.x;
                nm[2 * g + 1] = v.y;
            }
        };
        auto clear_row = [&](uint8_t* at) {      // its column blocks l4, l4 + 4: whether it holds (or held) an infinity or NaN
            bool cleared = false;
#pragma unroll 1
            for (int cb = l4; cb < n_cb; cb += 4)
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                    uint4* piece = reinterpret_cast<uint4*>(at + (size_t)cb * kTBlk + 16 * k);
                    const uint4 v = *piece;
                    const uint4 w = make_uint4(finite_pair(v.x, cleared), finite_pair(v.y, cleared), finite_pair(v.z, cleared),
                                               finite_pair(v.w, cleared));
                    *piece = w;
                }
            return cleared;
        };
        int hv[8] = {};              // kPack: which rows each of the thread's heads sees
        // i0: this thread's first row of the list
        auto softmax = [&](const Run& run, int i0, bool first) {
            const uint32_t buf = n & 1u;
            mwait(&tl->full[buf][0], (n >> 1) & 1u);   // (long before S^T: makes `valid` visible)
            const uint32_t val = *reinterpret_cast<const uint16_t*>(&tl->valid[buf][2 * qd]) >> (lane >> 2);
            mwait(&tl->s_full[buf], (n >> 1) & 1u);
            tc_fence_after();
            const uint32_t ts = tmem + lane_base + 64u * buf + 32u * (uint32_t)set;
            uint32_t r[16];
            tmem_ld_rows16(ts, r);
            const bool v0 = (val & 1u) && !dead, v1 = (val & 0x100u) && !dead;
            auto sees = [&](int i, int second) {   // the thread's head i its first or second row
                const bool v = second ? v1 : v0;
                if (!kPack) return v;
                const int at = i0 + 8 * second;
                return v && at < run.n - (hv[i] >> 8) && (at >= run.nf + (hv[i] & 255) || at < p.n_first);
            };
            tmem_ld_wait();
            if (kPack) {
                // A row with an infinity or NaN has such scores with every head: NaN for those that see it, and something finite in
                // their place in the tile, so that P = 0 keeps them from the others.  (A finite row's score may pass fp32 too.)
                bool bad0 = false, bad1 = false;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const bool b = (r[k] & 0x7F800000u) == 0x7F800000u;
                    if (k & 2) bad1 = bad1 || b;
                    else bad0 = bad0 || b;
                }
                if (__any_sync(kWarpFull, bad0 || bad1)) {
                    mwait(&tl->full[buf][kHalves - 1], (n >> 1) & 1u);   // (complete: makes the rows visible)
                    auto holds = [&](bool bad, int at) {   // four lanes have a quarter of the row each
                        const uint32_t lanes = 0xFu << (lane & 28);
                        const bool look = (__ballot_sync(kWarpFull, bad) & lanes) != 0;
                        return (__ballot_sync(kWarpFull, look && clear_row(t_s + buf * kTile + at * 128)) & lanes) != 0;
                    };
                    bad0 = holds(bad0, row);
                    bad1 = holds(bad1, row + 8);
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (k & 2 ? bad1 : bad0) r[k] = 0x7FFFFFFFu;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) saw |= (sees(i, 0) || sees(i, 1)) ? 1u << i : 0u;
            } else {
                saw |= v0 || v1 ? 0xFFu : 0u;
            }
            float y[16];
            float top0 = -INFINITY, top1 = -INFINITY;
            auto scale = [&]() {
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[4 * g + k] = fmaf(__uint_as_float(r[4 * g + k]), c, nm[2 * g + (k & 1)]);
            };
            scale();
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (kPack) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (sees(2 * g + (k & 1), k >> 1)) top0 = fmaxf(top0, y[4 * g + k]);
                } else {
                    top0 = fmaxf(top0, fmaxf(y[4 * g], y[4 * g + 1]));
                    top1 = fmaxf(top1, fmaxf(y[4 * g + 2], y[4 * g + 3]));
                }
            }
            // the references stay unless a visible score passes its head's by 2^8 or a head has none yet (of a run's first tile
            // it may see no row: pages outside the pool)
            const bool need = !named_bar_and(bar_set, 128, !(first || unset || ((kPack || v0) && top0 > kTopMost) || (v1 && top1 > kTopMost)));
            if (need) {
                float* red = &tl->red[buf][set][qd][0];
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = fmaxf(sees(i, 0) ? y[4 * (i >> 1) + (i & 1)] : -INFINITY,
                                 sees(i, 1) ? y[4 * (i >> 1) + 2 + (i & 1)] : -INFINITY);
                red[own_head] = over_rows<true>(v);
                named_bar_sync(bar_set, 128);
                const float* rr = &tl->red[buf][set][0][lane];
                float* own = &tl->neg_m[set][qd][0];
                const float mt = fmaxf(fmaxf(rr[0], rr[32]), fmaxf(rr[64], rr[96])) - own[lane];
                const float m_new = (m_run == -INFINITY || mt > m_run + kTopMost) ? fmaxf(m_run, mt) : m_run;
                const float alpha = (m_new == m_run) ? 1.f : fast_exp2(m_run - m_new);
                m_run = m_new;
                unset = __any_sync(kWarpFull, m_new == -INFINITY && 32 * set + lane < run.heads);
                __syncwarp();
                // a head without any finite score keeps -inf; its exponents are taken from 0, so that NaN
                // scores show in its output
                own[lane] = m_new == -INFINITY ? 0.f : -m_new;
                __syncwarp();
                load_m();
                scale();
                if (!first && !dead && __any_sync(kWarpFull, alpha != 1.f)) {
                    mwait(&tl->freed[buf ^ 1u][kHalves - 1], ((n - 1) >> 1) & 1u);   // the previous tile's PV is done
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < 2 * NM; ++k) {
                        const uint32_t ta = tmem + lane_base + o_block(runs - 1, (uint32_t)k >> 1) + 32u * (uint32_t)set + 16u * (k & 1);
                        uint32_t o[16];
                        tmem_ld16(ta, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * __shfl_sync(kWarpFull, alpha, 16 * (k & 1) + i));
                        tmem_st16(ta, o);
                    }
                    tmem_st_wait();
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        l_thr[2 * g] *= __shfl_sync(kWarpFull, alpha, 8 * g + 2 * l4);
                        l_thr[2 * g + 1] *= __shfl_sync(kWarpFull, alpha, 8 * g + 2 * l4 + 1);
                    }
                }
            }
            uint8_t* prow = p_s + buf * kPBuf + row * 128 + 4 * l4;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float a0 = sees(2 * g, 0) ? fast_exp2(y[4 * g]) : 0.f, a1 = sees(2 * g + 1, 0) ? fast_exp2(y[4 * g + 1]) : 0.f;
                const float b0 = sees(2 * g, 1) ? fast_exp2(y[4 * g + 2]) : 0.f, b1 = sees(2 * g + 1, 1) ? fast_exp2(y[4 * g + 3]) : 0.f;
                l_thr[2 * g] += a0 + b0;
                l_thr[2 * g + 1] += a1 + b1;
                const int at = ((4 * set + g) ^ (row & 7)) << 4;
                *reinterpret_cast<uint32_t*>(prow + at) = pack_bf16x2(a0, a1);
                *reinterpret_cast<uint32_t*>(prow + 8 * 128 + at) = pack_bf16x2(b0, b1);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tl->p_full[buf]);
        };

        // The end of a run: its heads' sums, lse and factors, or for a partial (slot >= 0) sums and references.
        auto finish = [&](const Run& run, float sink, float prev_lse) {
            uint32_t any = saw;
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) any |= __shfl_xor_sync(kWarpFull, any, o);
            // the sum of a head that saw none of the rows is -0, which adds up to -0 over such parts alone
            const float sum = over_rows<false>(l_thr);
            tl->lsum[set][qd][own_head] = any >> own_i & 1u ? sum : -0.f;
            named_bar_sync(bar_set, 128);
            if (qd != 0) return;
            const float* ls = &tl->lsum[set][0][lane];
            const float lt = (ls[0] + ls[32]) + (ls[64] + ls[96]);
            const int hh = 32 * set + lane;
            float inv = 0.f, wp = 0.f;
            if (run.slot >= 0) {
                p.part_ml[run.slot * 64 + hh] = make_float2(m_run, lt);
            } else if (signbit(lt) && hh < run.heads) {
                // a query that sees no row: what it had
                wp = prev_lse == -INFINITY ? 0.f : 1.f;
                if (p.lse) p.lse[run.row0 + hh] = prev_lse;
            } else if (hh < run.heads) {
                // everything relative to the largest of the reference, the sink and prev_lse
                const float sk = sink * kLog2e, pl = prev_lse * kLog2e;
                float mx = fmaxf(m_run, fmaxf(sk, pl));
                if (mx == -INFINITY) mx = 0.f;
                const float f = lt == 0.f ? 0.f : fast_exp2(m_run - mx);   // (without a reference lt is 0 or NaN)
                const float ep = fast_exp2(pl - mx);
                const float den = lt * f + fast_exp2(sk - mx) + ep;
                const float over = __fdividef(1.f, den);
                inv = f * over;
                wp = ep * over;
                if (p.lse) p.lse[run.row0 + hh] = (mx + __log2f(den)) * kLn2;
            }
            // (this run's scores mean that a PV of the run two before is done, and so that the run four before has been written)
            const uint32_t k = (runs - 1) % kRuns;
            tl->fac[k][hh] = make_float2(inv, wp);
            __syncwarp();
            if (lane == 0) mbar_arrive(&tl->fac_full[k]);
        };

        Run run;
        const int hh = 32 * set + lane;
        const float sink = p.sink && hh < hp ? __ldg(p.sink + hh % p.h) : -INFINITY;
        uint32_t par = 0;                      // run parity
        while (next_run(run, true)) {
            // (not by __ldg: the kernel before, which may have written it, can still run when this one starts)
            const float prev_lse = p.prev_lse && qd == 0 && hh < run.heads ? __ldcg(p.prev_lse + run.row0 + hh) : -INFINITY;
            if (kPack) {
                if (tid < 64) tl->vis[par][tid] = head_vis(p, run, tid);   // (every warp is done with par's last)
                named_bar_sync(kBarSoft, 256);
#pragma unroll
                for (int i = 0; i < 8; ++i) hv[i] = tl->vis[par][32 * set + 8 * (i >> 1) + 2 * l4 + (i & 1)];
            }
            m_run = -INFINITY;
            tl->neg_m[set][qd][lane] = 0.f;
            __syncwarp();
            load_m();
#pragma unroll
            for (int i = 0; i < 8; ++i) l_thr[i] = 0.f;
            saw = 0;
            unset = false;
            for (int t = run.t0; t < run.t1; ++t, ++n)
                if (active) softmax(run, t * kRows + row, t == run.t0);
            if (active) finish(run, sink, prev_lse);
            par ^= 1u;
        }

        // queries past the table are reported; groups whose lists are empty
        for (int q = blockIdx.x; q < nq; q += gridDim.x) {
            const PagedGroup grp = group_of(p, q);
            if (tid == 0 && grp.heads > 0 && p.status &&
                (uint32_t)__ldg(p.start_pos + grp.b) + (uint32_t)(grp.t0 + grp.heads / p.h) > (uint32_t)p.cap)
                atomicOr(p.status, 1u /* STI_FLAG_INDEX_RANGE */);
            if (group_rows(p, grp.b, q - grp.b * p.groups) > 0) continue;
            if (tid == 0 && p.by_query) p.rec[q] = make_int2(-1, 0);
            for (int i = tid; i < grp.heads; i += 256)
                if (p.lse) p.lse[grp.row0 + i] = p.prev_lse ? p.prev_lse[grp.row0 + i] : -INFINITY;
            const int chunks = p.d / 8;
#pragma unroll 4
            for (int i = tid; i < grp.heads * chunks; i += 256) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (p.prev_out) {
                    v = reinterpret_cast<const uint4*>(p.prev_out + grp.row0 * p.d)[i];
                    if (p.prev_lse[grp.row0 + i / chunks] == -INFINITY) v = make_uint4(0, 0, 0, 0);
                }
                reinterpret_cast<uint4*>(p.out + grp.row0 * p.d)[i] = v;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort) {   // a wait gave up: let the MMAs and copies in flight finish before the CTA's memory goes
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 50000ull) {
        }
    }
    if (warp == kQkWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

// ------------------------------------------------------------------ joining split queries

// What a warp of the joining kernels has: four heads (lane l looks after head l % 4 of them) x 32 Q dims of a query, a lane
// dims lane + 32 j.  (Going through the code once before the wait, with nothing read or written, so that it is in the
// instruction cache: 118 -> 120 us for 32 queries over 16384 rows, since not all blocks are there that early.)
struct Quad {
    float mx, l, sink, prev_lse;   // of the lane's head: largest reference, sum relative to it; -inf: none
    bool seen;                     // it sees a row
};
__device__ __forceinline__ float over_parts_max(float v) {
#pragma unroll
    for (int o = 16; o >= 4; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kWarpFull, v, o));
    return v;
}
// The largest reference becomes that of the sink and prev_lse too.
__device__ __forceinline__ void quad_top(Quad& q, bool any) {
    q.seen = (__ballot_sync(kWarpFull, any) >> (threadIdx.x & 3) & 0x11111111u) != 0;
    if (!q.seen) q.sink = -INFINITY;
    q.mx = fmaxf(over_parts_max(q.mx), fmaxf(q.sink, q.prev_lse * kLog2e));
    if (q.mx == -INFINITY) q.mx = 0.f;
}
// This block's record, {-1, 0} if there is none: also where the attention gave up a wait and left anything (first: below n).
__device__ __forceinline__ int2 split_of(const AttnPagedParams& p, int n) {
    const int2 rec = __ldcg(p.rec + blockIdx.x);
    const int c = p.by_query ? rec.x : (int)blockIdx.x;
    return rec.x >= 0 && rec.x < n && rec.y > c && rec.y < p.grid ? rec : make_int2(-1, 0);
}
// The factor of a part.  One of which the head sees nothing has a sum of -0 and O = 0; one without a finite score has no
// reference, and a sum of 0 or NaN.
__device__ __forceinline__ float part_factor(const float2& ml, float mx) { return ml.y == 0.f ? 0.f : exp2f(ml.x - mx); }
__device__ __forceinline__ void add4(float4& o, const float4& w, const float4& v) {
    o.x += w.x * v.x;
    o.y += w.y * v.y;
    o.z += w.z * v.z;
    o.w += w.w * v.w;
}
// prev_out of the warp's heads and dims, from its first on.
template <int Q>
__device__ __forceinline__ void quad_prev(const AttnPagedParams& p, int64_t at, int there, int blocks, uint16_t (&pv)[Q][4]) {
#pragma unroll
    for (int j = 0; j < Q; ++j)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            pv[j][h] = 0;
            if (p.prev_out && j < blocks && h < there) pv[j][h] = p.prev_out[at + 32 * j + (int64_t)h * p.d];
        }
}
// lse (lse_at >= 0) and the outputs.
template <int Q>
__device__ __forceinline__ void quad_out(const AttnPagedParams& p, const Quad& q, int64_t lse_at, int64_t at, int there, int blocks,
                                         const float4 (&o)[Q], const uint16_t (&pv)[Q][4]) {
    const float pl = q.prev_lse * kLog2e, ep = exp2f(pl - q.mx), den = q.l + exp2f(q.sink - q.mx) + ep;
    if (lse_at >= 0) p.lse[lse_at] = q.seen ? (q.mx + log2f(den)) * kLn2 : q.prev_lse;
    // a query that sees no row keeps what it had
    const float inv = q.seen ? 1.f / den : 0.f, wp = q.seen ? ep / den : pl == -INFINITY ? 0.f : 1.f;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float f = __shfl_sync(kWarpFull, inv, h), w = __shfl_sync(kWarpFull, wp, h);
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            float x = (h == 0 ? o[j].x : h == 1 ? o[j].y : h == 2 ? o[j].z : o[j].w) * f;
            if (w != 0.f) x += w * __uint_as_float((uint32_t)pv[j][h] << 16);   // weight 0: prev_out is not used
            if (j < blocks && h < there) p.out[at + 32 * j + (int64_t)h * p.d] = __bfloat16_as_ushort(__float2bfloat16(x));
        }
    }
}

// Few parts: a warp adds them up in order, U at a time (block (x, y): warps 8 y ... of a query).  kByQuery: x is the
// query, of which p.rec says whether it is split.  Otherwise, when there are more queries than CTAs, most CTAs' last query
// is: x is the CTA, and the first U parts are on their way before it is known whether there are any.
template <int U, bool kByQuery>
__global__ void __launch_bounds__(256) merge_few_kernel(const AttnPagedParams p) {
    const int lane = threadIdx.x & 31, quads = (p.pack * p.h + 3) / 4, unit = (int)blockIdx.y * 8 + ((int)threadIdx.x >> 5);
    const int m = unit / quads, quad = unit - m * quads, blocks = min(4, p.d / 32 - 4 * m);
    const int hd = 4 * quad + (lane & 3), own = lane >> 2;   // the lane's head, and its part of 8 at a time
    griddep_launch_dependents();
    griddep_wait();
    if (blocks <= 0) return;
    const int2 rec = split_of(p, kByQuery ? p.grid : p.B * p.groups);
    if (kByQuery && rec.x < 0) return;
    const int c = kByQuery ? rec.x : (int)blockIdx.x;
    auto slot = [&](int i) { return i == 0 ? 2 * c + 1 : 2 * min(c + i, p.grid - 1); };   // (the last CTA's again past the end)
    const float4* src = reinterpret_cast<const float4*>(p.part_o) + (4 * m * quads + quad) * 32 + lane;
    const float2* stats = p.part_ml + hd;
    float4 v[U][4];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j < blocks) v[k][j] = __ldcg(src + (int64_t)slot(i0 + k) * p.d * quads + j * quads * 32);
            }
    };
    float2 ml = __ldcg(stats + slot(own) * 64);
    load(0);
    if (rec.x < 0) return;
    const PagedGroup grp = group_of(p, kByQuery ? (int)blockIdx.x : rec.x);
    const int there = grp.heads - 4 * quad, parts = rec.y - c + 1;
    if (there <= 0) return;
    const bool mine = (lane & 3) < there;
    const int64_t at = (grp.row0 + 4 * quad) * p.d + 128 * m + lane;
    uint16_t pv[4][4];
    quad_prev(p, at, there, blocks, pv);
    Quad q{-INFINITY, 0.f, p.sink && mine ? __ldg(p.sink + hd % p.h) * kLog2e : -INFINITY,
           p.prev_lse && mine ? p.prev_lse[grp.row0 + hd] : -INFINITY, false};
    bool any = false;
    for (int i = own; i < parts; i += 8) {
        if (i >= 8) ml = __ldcg(stats + slot(i) * 64);
        any = any || !signbit(ml.y);
        q.mx = fmaxf(q.mx, ml.x);
    }
    quad_top(q, any);
    float f = 0.f;
    float4 o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0;;) {
        if ((i0 & 7) == 0) {   // the factors of parts i0 .. i0 + 7
            if (parts > 8 && i0 + own < parts) ml = __ldcg(stats + slot(i0 + own) * 64);
            f = i0 + own < parts ? part_factor(ml, q.mx) : 0.f;
            q.l += i0 + own < parts ? ml.y * f : 0.f;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int from = ((i0 + k) & 7) * 4;
            const float4 w = make_float4(__shfl_sync(kWarpFull, f, from), __shfl_sync(kWarpFull, f, from + 1),
                                         __shfl_sync(kWarpFull, f, from + 2), __shfl_sync(kWarpFull, f, from + 3));
            if (i0 + k < parts)
#pragma unroll
                for (int j = 0; j < 4; ++j) add4(o[j], w, v[k][j]);
        }
        i0 += U;
        if (i0 >= parts) break;
        load(i0);
    }
#pragma unroll
    for (int s = 16; s >= 4; s >>= 1) q.l += __shfl_xor_sync(kWarpFull, q.l, s);
    quad_out(p, q, p.lse && m == 0 && lane < 4 && mine ? grp.row0 + hd : -1, at, there, blocks, o, pv);
}

// Queries of many parts, by query: G warps take every G-th part; the first of them works the factors out while everyone's
// first parts are on their way, and adds up the warps' sums in order.
template <int G, int Q>
__global__ void __launch_bounds__(256) merge_many_kernel(const AttnPagedParams p) {
    constexpr int U = 4, kUnits = 8 / G, kMost = 160;   // parts in flight; units per block; parts, at most
    __shared__ float4 fac[kUnits][kMost];
    __shared__ float4 sums[8][Q][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = warp % G, own_unit = warp / G;
    const int quads = (p.pack * p.h + 3) / 4, unit = (int)blockIdx.y * kUnits + own_unit;
    const int m = unit / quads, quad = unit - m * quads, blocks = min(Q, p.d / 32 - Q * m);   // none past the last unit
    const int hd = 4 * quad + (lane & 3), own = lane >> 2;
    griddep_launch_dependents();
    griddep_wait();
    const int2 rec = split_of(p, p.grid);
    if (rec.x < 0) return;
    const int c = rec.x, parts = rec.y - c + 1;
    auto slot = [&](int i) { return i == 0 ? 2 * c + 1 : 2 * (c + min(i, parts - 1)); };   // (the last one again past the end)
    const float4* src = reinterpret_cast<const float4*>(p.part_o) + (Q * m * quads + quad) * 32 + lane;
    float4 v[U][Q];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int j = 0; j < Q; ++j) {
                v[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j < blocks) v[k][j] = __ldcg(src + (int64_t)slot(i0 + k * G) * p.d * quads + j * quads * 32);
            }
    };
    load(g);
    const PagedGroup grp = group_of(p, (int)blockIdx.x);
    const int there = blocks > 0 ? grp.heads - 4 * quad : 0;
    const bool mine = (lane & 3) < there;
    const int64_t at = (grp.row0 + 4 * quad) * p.d + 32 * Q * m + lane;
    Quad q{-INFINITY, 0.f, -INFINITY, -INFINITY, false};
    uint16_t pv[Q][4];
    if (g == 0) {
        const float2* stats = p.part_ml + hd;
        float2 ml[kMost / 8];
#pragma unroll
        for (int k = 0; k < kMost / 8; ++k) {
            if (8 * k >= parts) break;
            ml[k] = own + 8 * k < parts ? __ldcg(stats + slot(own + 8 * k) * 64) : make_float2(-INFINITY, -0.f);
        }
        quad_prev(p, at, there, blocks, pv);
        if (p.sink && mine) q.sink = __ldg(p.sink + hd % p.h) * kLog2e;
        if (p.prev_lse && mine) q.prev_lse = p.prev_lse[grp.row0 + hd];
        bool any = false;
#pragma unroll
        for (int k = 0; k < kMost / 8; ++k) {
            if (8 * k >= parts) break;
            any = any || !signbit(ml[k].y);
            q.mx = fmaxf(q.mx, ml[k].x);
        }
        quad_top(q, any);
#pragma unroll
        for (int k = 0; k < kMost / 8; ++k) {
            if (8 * k >= parts) break;
            if (own + 8 * k < parts) {
                const float f = part_factor(ml[k], q.mx);
                reinterpret_cast<float*>(&fac[own_unit][own + 8 * k])[lane & 3] = f;
                q.l += ml[k].y * f;
            }
        }
#pragma unroll
        for (int o = 16; o >= 4; o >>= 1) q.l += __shfl_xor_sync(kWarpFull, q.l, o);
    }
    __syncthreads();
    float4 o[Q];
#pragma unroll
    for (int j = 0; j < Q; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = g; i0 < parts; i0 += U * G) {
        if (i0 != g) load(i0);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i0 + k * G >= parts) break;
            const float4 w = fac[own_unit][i0 + k * G];
#pragma unroll
            for (int j = 0; j < Q; ++j) add4(o[j], w, v[k][j]);
        }
    }
#pragma unroll
    for (int j = 0; j < Q; ++j) sums[warp][j][lane] = o[j];
    __syncthreads();
    if (g != 0) return;
#pragma unroll
    for (int j = 0; j < Q; ++j)
#pragma unroll
        for (int k = 1; k < G; ++k) {
            const float4 x = sums[warp + k][j][lane];
            o[j] = make_float4(o[j].x + x.x, o[j].y + x.y, o[j].z + x.z, o[j].w + x.w);
        }
    quad_out(p, q, p.lse && m == 0 && lane < 4 && mine ? grp.row0 + hd : -1, at, there, blocks, o, pv);
}

}  // namespace

template <int NM>
cudaError_t launch_attn_paged_nm(const CUtensorMap& tm_q, const AttnPagedParams& p, cudaStream_t stream) {
    const int nq = p.B * p.groups;
    const size_t smem = attn_paged_smem(p.d);
    const int kind = 4 * (p.groups == 1) + 2 * (p.pack > 1) + (p.prev_out != nullptr);
    using Kernel = void (*)(CUtensorMap, AttnPagedParams);
    static constexpr Kernel kKernels[8] = {
        attn_paged_kernel<NM, false, false, false>, attn_paged_kernel<NM, false, true, false>,
        attn_paged_kernel<NM, true, false, false>,  attn_paged_kernel<NM, true, true, false>,
        attn_paged_kernel<NM, false, false, true>,  attn_paged_kernel<NM, false, true, true>,
        attn_paged_kernel<NM, true, false, true>,   attn_paged_kernel<NM, true, true, true>};
    const Kernel kernel = kKernels[kind];
    // The kernel's shared-memory limit, once per device (it follows from NM alone, so no other call asks for another).
    static std::atomic<uint64_t> set[8];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(set[kind].load(std::memory_order_acquire) & bit)) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
        set[kind].fetch_or(bit, std::memory_order_release);
    }
    e = launch_after(kernel, dim3((unsigned)p.grid), kPThreads, smem, stream, tm_q, p);
    if (e != cudaSuccess || p.whole) return e;
    // Parts of a query when they are alike.  A long one among short ones gets the short ones' join: one of 65536 rows x 512 among 63 of
    // 512 takes 62 us for the call, alone 29.
    const int parts = p.grid / nq + 1;
    const int quads = (p.pack * p.h + 3) / 4;
    auto grid = [&](int warps, int dims) {   // warps of four heads x dims, of each query that may be split
        return dim3((unsigned)(nq < p.grid ? nq : p.grid), (unsigned)((quads * ((p.d + dims - 1) / dims) * warps + 7) / 8));
    };
    return parts > 16   ? launch_after(merge_many_kernel<8, 2>, grid(8, 64), 256, 0, stream, p)
           : parts > 8  ? launch_after(merge_many_kernel<2, 4>, grid(2, 128), 256, 0, stream, p)
           : parts > 4  ? launch_after(merge_few_kernel<4, true>, grid(1, 128), 256, 0, stream, p)
           : p.by_query ? launch_after(merge_few_kernel<2, true>, grid(1, 128), 256, 0, stream, p)
                        : launch_after(merge_few_kernel<2, false>, grid(1, 128), 256, 0, stream, p);
}

}  // namespace sti
