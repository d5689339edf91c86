// tern_delta_chunk.cu -- the gated delta rule over prompts, 64 tokens at a time,
// on the tcgen05 tensor cores.
//
// With G the running sum of the decays' logs in a chunk and S the state before it,
//   A_ij = beta_i e^(G_i - G_j) k_i.k_j (j < i),   T = (I + A)^-1,
//   X = beta (V - e^G K S^T),   U = T X,
//   O = scale e^G Q S^T + P U,   P_ij = scale e^(G_i - G_j) q_i.k_j (j <= i),
//   S <- e^(G_last) S + sum_j e^(G_last - G_j) u_j k_j^T.
// A CTA takes 128 rows of one head's S through its sequence.  Everything with rows
// of S (S itself, X, U, O) is kept transposed, a tensor memory lane a row, so those
// products have M = 128 and their left operand in tensor memory, and what passes
// from one product to the next never leaves its lane.
//
// What bounds a sequence is the chain from chunk to chunk, three phases of sixteen
// warps (four threads a row) between three products:
//   S = e^G_last S + D, its parts to tensor memory  ->  [K; Q] S^T
//   X                                               ->  U = T X
//   e^(G_last - G) U                                ->  D = U^T K
// and beside it: P U; four warps for the output; the Gram matrices [K; Q] K^T of the
// chunk after the next, from which four warps make P and T (16 x 16 blocks by
// substitution, a column a lane, joined by mma.sync); two for decays and lengths.
//
// A chunk takes 4.0 us where few SMs run, 4.6 where all do (latency of that chain, the
// issue of some 17 thousand instructions by 32 warps, and, with all SMs at work, the
// fetching of code): six prompts, 16381 tokens of 48 heads of 128 x 128, 386 us, and one
// of 2048 tokens of 32 heads 138 us whole.  Where that leaves SMs idle, sequences go in
// pieces at once (DeltaPieces): 99 us.
//
// Rounding.  q, k, v are exact as bf16.  S, X, U, T and P are fp32 cut into two bf16
// values, which carry 2^-17 of each (one would lose 2^-8 of the state a chunk); what
// that leaves of X is added to U in fp32, T's diagonal being 1.  Lengths and decays
// are applied in fp32, to rows and columns of results.  Exponents are differences of G, at
// most 0, and G is a sum in 64 bits kept as two fp32: a long or strong decay before
// a pair of tokens does not blur theirs.
//
// A value that is not finite would reach back: T and P are 0 above their diagonals, and
// 0 x NaN is NaN.  It also stays in its rows of S for good, so those that are not finite
// at the end go once more, token by token, up to where they are not (redo): no code in the
// loops above (masks in X and A took 8 % of the time where sequences go in pieces).
#include "tern_delta.cuh"
#include "tern_sm100.cuh"

namespace tern {
namespace {

using namespace sm100;

__device__ int g_delta_chunk_error;

constexpr int kTok = kDeltaChunk, kRows = kDeltaRows;                 // tokens of a chunk, rows of S
constexpr int kKqStages = 3, kVStages = 2, kCoefStages = 4, kTpStages = 2, kAStages = 2;
constexpr uint32_t kTile = kTok * 128;                // bytes of a [64][64] bf16 tile, 128-byte swizzled rows
constexpr uint32_t kATile = kTok * 64;                // of a part of A below its diagonal blocks: a_at()
// P's two parts, side by side in rows of 64 values: columns 0 .. 31 of all 64 tokens, then 32 .. 63
// of the later 32 (the earlier have none)
constexpr uint32_t kPRight = kTile, kPBytes = kTile + kTile / 2;
constexpr int kDiagRow = 20, kDiagBlock = 16 * kDiagRow + 16;   // floats of a column and of a block of -A's diagonal blocks

// What one chunk's tokens are scaled by.
struct alignas(16) Coef {
    float beta[kTok], near[kTok];   // beta; e^G
    float minus_near[kTok];         // -beta e^G |k|^-1
    float left[kTok];               // e^(G_last - G) |k|^-1
    float near_q[kTok];             // scale e^G |q|^-1
    float scale_q[kTok];            // scale |q|^-1
    float to_end[kTok];             // |k|^-1 e^(G at its 16's last token - G)
    float2 G[kTok];                 // G in powers of two, two parts
    float2 Gk[kTok];                // G - log |k|^-1
    float2 end[4];                  // that of each 16's last token
    float last, unused[3];          // e^G_last
};

template <int DK>
struct Cfg {
    static constexpr int NC = DK / 64;                          // chunks of 64 values of a K or Q row
    static constexpr int COLS = DK / 4;                         // columns of S that a thread holds
    static constexpr int kKqBytes = NC * 2 * (int)kTile;        // 64 values of K's and Q's rows, the next 64
    static constexpr int kVBytes = 4 * kTok * 64;               // 32 rows of S a tile: [token][32]
    static constexpr int kTpBytes = 2 * (int)kTile + (int)kPBytes;   // T's two parts, P's
    static constexpr int kABytes = 2 * (int)kATile + 4 * kDiagBlock * 4;   // A's two parts, its diagonal blocks
    static constexpr size_t kKq = 0, kV = kKq + (size_t)kKqStages * kKqBytes, kTp = kV + (size_t)kVStages * kVBytes,
                            kA = kTp + (size_t)kTpStages * kTpBytes, kCoef = kA + (size_t)kAStages * kABytes, kBar = kCoef + kCoefStages * sizeof(Coef),
                            kMisc = kBar + 48 * 8, kSmem = kMisc + 128 + 1024;
};
// warps: the chain, the output, A and P, T, then one each for products and copies and two for decays
constexpr int kOutWarp = 16, kGramWarp = 20, kInvWarp = 24, kMmaWarp = 28, kTmaWarp = 29, kCoefWarp = 30, kThreads = 32 * 32;
// registers a thread: 512 x 72 + 128 x (56 + 64 + 56 + 48) = 1024 x 64, what the CTA is launched with
// tensor memory columns: D over the parts of S; Q S^T of odd chunks; K S^T, then U, then U's parts; Q S^T
// of even chunks; the parts of X, then of the scaled U (X cannot take the place of S, which Q S^T may
// still be read from when K S^T is there); P U; Gram matrices
enum { T_S = 0, T_QS_ODD = 128, T_KS = 192, T_QS_EVEN = 256, T_X = 320, T_UP = T_X, T_O = 384, T_GRAM = 448 };
enum {
    KQ_FULL = 0, KQ_EMPTY = KQ_FULL + kKqStages, V_FULL = KQ_EMPTY + kKqStages, V_EMPTY = V_FULL + kVStages,
    COEF_FULL = V_EMPTY + kVStages, COEF_EMPTY = COEF_FULL + kCoefStages, TP_FULL = COEF_EMPTY + kCoefStages,
    TP_EMPTY = TP_FULL + kTpStages, GRAM_FULL = TP_EMPTY + kTpStages, GRAM_EMPTY, KS_FULL, U_FULL, D_FULL, O_FULL, O_EMPTY, A_FULL, A_EMPTY = A_FULL + kAStages, LENGTHS = A_EMPTY + kAStages,
    INVERSE, DIAG_FULL, TAIL = DIAG_FULL + kAStages, DRAIN, BARS
};
static_assert(BARS <= 48, "barriers");
// From the chain's 16 warps to the one that issues products: the SM's own barriers, whose
// last arrival wakes it sooner than an mbarrier's.  Nothing bounds a wait at one, so both
// sides go through all their turns whatever has failed, and no warp may be a turn ahead: it
// would be counted in another's place, and the last turn would miss one.  A warp of the chain
// is held by its waits (each turn's product is issued after the turn); one of which a wait has
// given up waits for nothing more, and goes through what is left at the barriers themselves.
enum { S_READY = 1, X_READY, UP_READY, U2_READY, TURNS = 4 };
constexpr int kChainThreads = 512 + 32;
__device__ __forceinline__ void chain_arrive(int b) { asm volatile("bar.arrive %0, %1;" ::"r"(b), "n"(kChainThreads) : "memory"); }
__device__ __forceinline__ void chain_wait(int b) { asm volatile("bar.sync %0, %1;" ::"r"(b), "n"(kChainThreads) : "memory"); }
// The chain's warps alone; true if `x` is, of any thread.
__device__ __forceinline__ void chain_sync() { asm volatile("bar.sync 5, 512;" ::: "memory"); }
__device__ __forceinline__ bool chain_any(bool x) {
    uint32_t any;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.or.pred q, 5, 512, p;\nselp.u32 %0, 1, 0, q;\n}" : "=r"(any) : "r"((uint32_t)x) : "memory");
    return any != 0;
}
__device__ __forceinline__ void chain_rest(int turn, int chunks) {   // the turns from `turn` on
#pragma unroll 1
    for (; turn < TURNS * chunks; ++turn) chain_wait(S_READY + turn % TURNS);
}

__device__ __forceinline__ int bar_count(int i) {
    if (i >= V_EMPTY && i < V_EMPTY + kVStages) return 4;
    if ((i >= COEF_FULL && i < COEF_EMPTY) || (i >= DIAG_FULL && i < TAIL)) return 2;
    if (i >= COEF_EMPTY && i < TP_FULL) return 20;
    if ((i >= TP_FULL && i < TP_EMPTY) || i == GRAM_EMPTY || i == O_EMPTY || (i >= A_FULL && i <= INVERSE)) return 4;
    return 1;
}

// A 16-byte unit of a row of a tile of 64 bf16 a row with 128-byte swizzled rows.
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int row, int unit) {
    return tile + (uint32_t)(row * 128 + ((unit ^ (row & 7)) << 4));
}
__device__ __forceinline__ void ldsm2_t(uint32_t& a, uint32_t& b, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}
// an 8 x 8 bf16 matrix, a row over four lanes, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Column `col` of the inverse of a 16 x 16 unit lower triangle, whose negated strict
// part lies at A by columns: each value found is at once taken to all below it.
__device__ __forceinline__ void solve16(const float* A, int col, float (&t)[16]) {
    uint64_t pair[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) pair[i] = pack2(2 * i == col ? 1.0f : 0.0f, 2 * i + 1 == col ? 1.0f : 0.0f);
#pragma unroll
    for (int i = 0; i < 15; ++i) {
        float x, y;
        unpack2(pair[i / 2], x, y);
        const uint64_t f = (i & 1) ? pack2(y, y) : pack2(x, x);
#pragma unroll
        for (int r = i / 4; r < 4; ++r) {
            const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(A + i * kDiagRow + 4 * r);
            if (4 * r + 1 > i) pair[2 * r] = fma2(f, a.x, pair[2 * r]);
            pair[2 * r + 1] = fma2(f, a.y, pair[2 * r + 1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) unpack2(pair[i], t[2 * i], t[2 * i + 1]);
}
// Where 8 columns of a row of A below its diagonal blocks stand: 32 columns a row; those of
// the second half's own block in the rows of the first 16, which have none.
__device__ __forceinline__ uint32_t a_at(uint32_t tile, int row, int unit) {
    return tile + (uint32_t)(row * 64 + ((unit ^ (row >> 1 & 3)) << 4));
}
// Rows R.., columns C.. of T below its diagonal blocks, 8 columns `n8` of it a warp:
//   -T22 (A21 T11),  T11 and T22 the 16 B rows from C and R on, every product of two
// parts each without the smallest (lo lo).
template <int B>
__device__ __forceinline__ void join_blocks(uint32_t A, uint32_t T, int R, int C, int n8, int lane) {
    const int a_row = C == 0 ? R : 0;
    float m[B][4];
#pragma unroll
    for (int i = 0; i < B; ++i) m[i][0] = m[i][1] = m[i][2] = m[i][3] = 0.0f;
#pragma unroll
    for (int kb = 0; kb < B; ++kb) {
        uint32_t bh[2], bl[2];
        const uint32_t at = tile_at(T, C + 16 * kb + (lane & 15), C / 8 + n8);
        ldsm2_t(bh[0], bh[1], at);
        ldsm2_t(bl[0], bl[1], at + kTile);
#pragma unroll
        for (int i = 0; i < B; ++i) {
            uint32_t ah[4], al[4];
            const uint32_t from = a_at(A, a_row + 16 * i + (lane & 15), 2 * kb + (lane >> 4));
            ldsm4(ah, from);
            ldsm4(al, from + kATile);
            mma_bf16(m[i], ah, bh[0], bh[1]);
            mma_bf16(m[i], ah, bl[0], bl[1]);
            mma_bf16(m[i], al, bh[0], bh[1]);
        }
    }
    uint32_t mh[B][2], ml[B][2];
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            uint32_t hi, lo;
            split2(-m[i][2 * x], -m[i][2 * x + 1], hi, lo);
            mh[i][x] = transpose8(hi);
            ml[i][x] = transpose8(lo);
        }
#pragma unroll
    for (int i = 0; i < B; ++i) {
        float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb <= i; ++kb) {
            uint32_t ah[4], al[4];
            const uint32_t from = tile_at(T, R + 16 * i + (lane & 15), R / 8 + 2 * kb + (lane >> 4));
            ldsm4(ah, from);
            ldsm4(al, from + kTile);
            mma_bf16(t, ah, mh[kb][0], mh[kb][1]);
            mma_bf16(t, ah, ml[kb][0], ml[kb][1]);
            mma_bf16(t, al, mh[kb][0], mh[kb][1]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            uint32_t hi, lo;
            split2(t[2 * x], t[2 * x + 1], hi, lo);
            const uint32_t to = tile_at(T, R + 16 * i + 8 * x + lane / 4, C / 8 + n8) + 4u * (lane & 3);
            sts32(to, hi);
            sts32(to + kTile, lo);
        }
    }
}

// The log of a decay in powers of two, times 2^40: |g| is at most 200 here.
__device__ __forceinline__ long long fixed_log2(float g) {
    g = g > 200.0f ? 200.0f : g;
    const float p = g * 1.44269502162933349609f, e = fmaf(g, 1.44269502162933349609f, -p) + g * 1.92596299e-8f;
    return __float2ll_rn(p * 1099511627776.0f) + __float2ll_rn(e * 1099511627776.0f);
}
__device__ __forceinline__ float unfixed(long long x) { return __ll2float_rn(x) * 9.094947017729282379e-13f; }

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)), "r"(src), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// the stores of this thread have read their shared memory; have been carried out
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// The sequence that comes `y`-th by length among its 32 neighbours: CTAs begin in their grid's
// order, and a long one that begins late is alone at the end.  Twelve prompts of 128 to 4096 tokens
// in no order, 48 heads, 461 -> 364 us; 32 short ones among which two are long 583 -> 439.
__device__ __forceinline__ int by_length(const StateSeqView& s, int y) {
    const int lane = threadIdx.x & 31, i = (y & ~31) + lane;
    const int mine = i < s.B ? max(s.q_start[i + 1] - s.q_start[i], 0) : -1;
    if (__all_sync(0xffffffffu, mine == __shfl_sync(0xffffffffu, mine, 0))) return y;
    int before = 0;   // (every lane another number)
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
        const int other = __shfl_sync(0xffffffffu, mine, j);
        before += other > mine || (other == mine && j < lane);
    }
    return (y & ~31) + __ffs(__ballot_sync(0xffffffffu, before == (y & 31))) - 1;
}

// What of a head a CTA has: the rows from row0 on of `rows`, the piece, whether it has the unit
// matrix in place of S.
struct Part {
    int h, row0, rows, piece;
    bool moves;
};
// S before the first token, of a thread's columns and row: the pool's, or a piece's
template <int DK>
__device__ __forceinline__ void first_state(const DeltaArgs& a, const StateSeq& s, const Part& p, float (&S)[DK / 4], int quarter, int row) {
    constexpr int COLS = DK / 4;
    if (p.piece > 0) {
#pragma unroll
        for (int i = 0; i < COLS; ++i) S[i] = p.moves && COLS * quarter + i == row ? 1.0f : 0.0f;
    } else {
        const float4* from = reinterpret_cast<const float4*>(
            a.state + (((long long)s.src * a.v_heads + p.h) * a.dv + p.row0 + row) * DK + COLS * quarter);
#pragma unroll
        for (int i = 0; i < COLS / 4; ++i) {
            const float4 x = s.src >= 0 && p.row0 + row < p.rows ? from[i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            S[4 * i] = x.x;
            S[4 * i + 1] = x.y;
            S[4 * i + 2] = x.z;
            S[4 * i + 3] = x.w;
        }
    }
}
// S after the last goes to the pool, or to where the join finds it: a sequence of more than one piece
template <int DK, bool PIECES>
__device__ __forceinline__ void last_state(const DeltaArgs& a, const StateSeq& s, const Part& p, const float (&S)[DK / 4], int quarter, int row) {
    constexpr int COLS = DK / 4;
    float* to_head = s.dst >= 0 && (s.n > 0 || s.dst != s.src) ? a.state + ((long long)s.dst * a.v_heads + p.h) * a.dv * DK : nullptr;
    unsigned char* parts = nullptr;
    if constexpr (PIECES) {
        const int all = load_state_seq(a.s, blockIdx.y, &g_delta_chunk_error).n;
        if (all > delta_piece_chunks(a.p, all) * kTok) {
            const long long at = (long long)blockIdx.y * a.v_heads + p.h;
            to_head = a.p.state + (at * a.p.count + p.piece) * ((long long)a.dv * DK);
            if (p.piece == 0) parts = delta_parts(a.p, blockIdx.y, a.v_heads, p.h, DK, (a.dv + kRows - 1) / kRows, p.row0 / kRows, 0);
            if (p.moves) parts = a.p.move + (at * (a.p.count - 1) + p.piece - 1) * delta_parts_bytes(DK, DK);
        }
        if (p.piece > 0 && s.n == 0) to_head = nullptr;
    }
    if (to_head) {
        float4* to = reinterpret_cast<float4*>(to_head + (p.row0 + row) * DK + COLS * quarter);
        if (!p.moves) {
#pragma unroll
            for (int i = 0; i < COLS / 4; ++i) to[i] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
        }
        if (PIECES && parts) {
#pragma unroll
            for (int i = 0; i < COLS; i += 8) put_parts8(parts, p.moves ? DK : kRows, DK, row, COLS * quarter + i, S + i);
        }
    }
}
__device__ __forceinline__ bool row_is_odd(const uint32_t* odd_rows, int w, int l) {
    return ((odd_rows[w & 3] | odd_rows[4 + (w & 3)] | odd_rows[8 + (w & 3)] | odd_rows[12 + (w & 3)]) >> l & 1u) != 0;
}
// Rows that are not finite at the end, token by token, by the chain's warps once the roles have met: a
// thread has its columns of its row again.  All is in shared memory, where the rings were: S by columns
// (a function has too few registers for it: 4.8 us a token, 2.2 so), a token's key, query, values and gates,
// and four partial sums a row.  Outputs are written over up to where a row is not finite.
template <int DK, bool PIECES>
__device__ __noinline__ void redo(const DeltaArgs& a, const StateSeq s, const Part p, const uint32_t* odd_rows, unsigned char* smem) {
    constexpr int COLS = DK / 4;
    constexpr int kBatch = 16;
    struct Staged {
        float S[DK][kRows];
        float k[kBatch][DK], q[kBatch][DK], v[kBatch][kRows];
        float4 gate[kBatch];
        float2 part[2][4][kRows];
    };
    static_assert(sizeof(Staged) <= Cfg<DK>::kBar, "in the place of the roles' rings");
    Staged& st = *reinterpret_cast<Staged*>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quarter = warp >> 2, row = (warp & 3) * 32 + lane;
    const bool mine = p.row0 + row < p.rows && row_is_odd(odd_rows, warp, lane);
    bool left = mine;   // still finite
    long long first_chunk = 0;   // of the piece's, in the outputs
    if (PIECES && p.piece > 0) {
        const StateSeq whole = load_state_seq(a.s, blockIdx.y, &g_delta_chunk_error);
        first_chunk = delta_piece_chunk(a.p.count, whole.t0, blockIdx.y) + (p.piece - 1) * delta_piece_chunks(a.p, whole.n);
    }
    float (*const S)[kRows] = reinterpret_cast<float (*)[kRows]>(&st.S[COLS * quarter][row]);   // this thread's: S[e][0]
    {
        float first[COLS], nothing = 0.0f;
        first_state<DK>(a, s, p, first, quarter, row);
#pragma unroll
        for (int e = 0; e < COLS; ++e) {
            S[e][0] = first[e];
            nothing = fmaf(first[e], 0.0f, nothing);
        }
        st.part[0][quarter][row] = make_float2(nothing, 0.0f);
        chain_sync();
        for (int i = 0; i < 4; ++i) left = left && st.part[0][i][row].x == 0.0f;
    }
#pragma unroll 1
    for (int t0 = 0; t0 < s.n; t0 += kBatch) {
        if (!chain_any(left)) break;
        const int n = min(kBatch, s.n - t0);
        if (warp < n) {
            const long long t = s.t0 + t0 + warp;
            delta_stage<DK>(a, t, p.h, lane, st.k[warp], st.q[warp], &st.gate[warp]);
            for (int i = lane; i < kRows; i += 32)
                st.v[warp][i] = !p.moves && p.row0 + i < p.rows ? __bfloat162float(a.v[t * a.v_token + (long long)p.h * a.dv + p.row0 + i]) : 0.0f;
        }
        chain_sync();
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const float4* k = reinterpret_cast<const float4*>(st.k[i] + COLS * quarter);
            const float4* q = reinterpret_cast<const float4*>(st.q[i] + COLS * quarter);
            float sk = 0.0f, sq = 0.0f;
#pragma unroll 4
            for (int e = 0; e < COLS / 4; ++e) {
                const float4 k4 = k[e], q4 = q[e];
                const float x = S[4 * e][0], y = S[4 * e + 1][0], z = S[4 * e + 2][0], w = S[4 * e + 3][0];
                sk = fmaf(x, k4.x, fmaf(y, k4.y, fmaf(z, k4.z, fmaf(w, k4.w, sk))));
                sq = fmaf(x, q4.x, fmaf(y, q4.y, fmaf(z, q4.z, fmaf(w, q4.w, sq))));
            }
            st.part[i & 1][quarter][row] = make_float2(sk, sq);
            chain_sync();   // (the other half of part is not written again before all have come to the next)
            sk = sq = 0.0f;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float2 two = st.part[i & 1][x][row];
                sk += two.x;
                sq += two.y;
            }
            const float4 gate = st.gate[i];
            const int token = t0 + i;
            const float u = gate.y * (st.v[i][row] - gate.x * sk), out = fmaf(u, gate.z, gate.x * sq);
#pragma unroll 4
            for (int e = 0; e < COLS / 4; ++e) {
                const float4 k4 = k[e];
                S[4 * e][0] = fmaf(u, k4.x, gate.x * S[4 * e][0]);
                S[4 * e + 1][0] = fmaf(u, k4.y, gate.x * S[4 * e + 1][0]);
                S[4 * e + 2][0] = fmaf(u, k4.z, gate.x * S[4 * e + 2][0]);
                S[4 * e + 3][0] = fmaf(u, k4.w, gate.x * S[4 * e + 3][0]);
            }
            if (left && quarter == 0) {
                if (!PIECES || p.piece == 0) {
                    a.out[((s.t0 + token) * (long long)a.v_heads + p.h) * a.dv + p.row0 + row] = __float2bfloat16(out);
                } else {
                    // as the output warps have it
                    const long long tile = (((first_chunk + token / kTok) * a.v_heads + p.h) * p.rows + p.row0) * (kTok * 4);
                    const int t = token % kTok;
                    if (p.moves) {
                        uint32_t hi, lo;
                        split2(out, 0.0f, hi, lo);
                        unsigned char* to = a.p.out_move + tile + row / 64 * (kTok * 128) + t * 128 + ((row % 64 / 8 ^ (t & 7)) << 4) + 2 * (row & 7);
                        *reinterpret_cast<unsigned short*>(to) = (unsigned short)hi;
                        *reinterpret_cast<unsigned short*>(to + DK * 128) = (unsigned short)lo;
                    } else {
                        reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(a.p.out) + tile)[t * min(kRows, p.rows - p.row0) + row] = out;
                    }
                }
            }
            left = left && fabsf(u) < INFINITY;
        }
    }
    if (mine) {
        float last[COLS];
#pragma unroll
        for (int e = 0; e < COLS; ++e) last[e] = left ? S[e][0] : NAN;
        last_state<DK, PIECES>(a, s, p, last, quarter, row);
    }
}

template <int DK, bool PIECES>
__global__ void __launch_bounds__(kThreads, 1)
delta_chunk_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_out,
                   const __grid_constant__ DeltaArgs a) {
    using C = Cfg<DK>;
    constexpr int NC = C::NC, COLS = C::COLS;
    extern __shared__ __align__(1024) unsigned char smem_dyn[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + (uint32_t)C::kBar + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
    uint32_t* const odd_rows = tmem_slot + 16;   // [chain's warps] rows of S that are not finite at the end, of its quarter
    Coef* const coefs = reinterpret_cast<Coef*>(smem + C::kCoef);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < BARS; ++i) mbar_init(bar(i), (uint32_t)bar_count(i));
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        tma_prefetch_desc(&tmap_out);
    }
    // T and P above their diagonal 16 x 16 blocks stay 0
    for (int i = threadIdx.x; i < kTpStages * C::kTpBytes / 16; i += kThreads)
        reinterpret_cast<uint4*>(smem + C::kTp)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;   // (all of it is this CTA's: it begins at 0)
    pdl_launch_dependents();
    pdl_wait();

    const int h = blockIdx.x % a.v_heads, row0 = blockIdx.x / a.v_heads * kRows, hk = h / a.group;
    // (every warp for itself: handed on through shared memory, the number costs the roles their uniform registers)
    const int b = !PIECES && a.by_length ? by_length(a.s, blockIdx.y) : (int)blockIdx.y;
    StateSeq s = load_state_seq(a.s, b, &g_delta_chunk_error);
    // this CTA's piece, whether it has the unit matrix in place of S, its rows
    int piece = 0, rows = a.dv;
    bool moves = false;
    if constexpr (PIECES) {
        const int z = blockIdx.z, per = delta_piece_chunks(a.p, s.n) * kTok;
        moves = z >= a.p.count;
        piece = moves ? z - a.p.count + 1 : z;
        if (moves) rows = DK;
        const int n = row0 < rows ? min(s.n - piece * per, per) : 0;
        s.t0 += piece * per;
        s.n = max(n, 0);
    }
    const Part part{h, row0, rows, piece, moves};
    const int chunks = (s.n + kTok - 1) / kTok;
    auto fail = [&] { report_device_error(&g_delta_chunk_error, TERN_DEVERR_DELTA_WAIT); };
    auto wait_warp = [&](int b, uint32_t parity) { return tern::wait_warp(bar(b), parity); };
    // the n-th use of a ring's stage: full, and free for it
    auto full = [](int n, int stages) { return (uint32_t)(n / stages) & 1u; };
    auto free = [](int n, int stages) { return ((uint32_t)(n / stages) & 1u) ^ 1u; };
    auto arrive = [&](int b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b));
    };

    if (warp < kOutWarp) {
        // ------------------------------ the chain ------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 72;");
        const int quarter = warp >> 2, row = (warp & 3) * 32 + lane;   // of S's columns and of a chunk's tokens
        const bool live = row0 + row < rows;
        const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = mine + T_S + (uint32_t)(COLS * quarter), tk = mine + T_KS + 16u * quarter;
        float S[COLS];
        first_state<DK>(a, s, part, S, quarter, row);
        // S = e^G_last S + D of a chunk; its parts in place of D
        auto next_state = [&](int c, bool more) {
            if (c >= 0) {
                if (!wait_warp(D_FULL, (uint32_t)c & 1u)) return false;
                tc_fence_after();
                const float last = coefs[c % kCoefStages].last;
                const uint64_t last2 = pack2(last, last);
                uint32_t d[COLS];
                if constexpr (COLS == 32) tmem_ld_x32(ts, d);
                else tmem_ld_x16(ts, d);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < COLS; e += 2)
                    unpack2(fma2(last2, pack2(S[e], S[e + 1]), pack2(__uint_as_float(d[e]), __uint_as_float(d[e + 1]))), S[e],
                            S[e + 1]);
            }
            if (more) {
                uint32_t hi[COLS / 2], lo[COLS / 2];
#pragma unroll
                for (int e = 0; e < COLS / 2; ++e) split2(S[2 * e], S[2 * e + 1], hi[e], lo[e]);
                if constexpr (COLS == 32) {
                    tmem_st_x16(ts, hi);
                    tmem_st_x16(ts + COLS / 2, lo);
                } else {
                    tmem_st_x8(ts, hi);
                    tmem_st_x8(ts + COLS / 2, lo);
                }
                tmem_st_wait();
                tc_fence_before();
                chain_arrive(S_READY);
            }
            if (c >= 0) arrive(COEF_EMPTY + c % kCoefStages);
            return true;
        };
        // -1, or the turns that have been gone through when a wait gave up
        auto walk = [&] {
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const uint32_t ph = (uint32_t)c & 1u;
                const Coef& k = coefs[c % kCoefStages];
                if (!next_state(c - 1, true)) return TURNS * c;
                if (!wait_warp(TP_FULL + (c & 1), full(c, kTpStages))) return TURNS * c + 1;
                float x[16];
                if (!wait_warp(V_FULL + c % kVStages, full(c, kVStages))) return TURNS * c + 1;
                const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(
                    smem + C::kV + (c % kVStages) * C::kVBytes + (warp & 3) * (kTok * 64) + quarter * (16 * 64)) + lane;
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const ulonglong2 beta = *reinterpret_cast<const ulonglong2*>(&k.beta[16 * quarter + i]);
                    unpack2(mul2(pack2(__bfloat162float(v[32 * i]), __bfloat162float(v[32 * i + 32])), beta.x), x[i], x[i + 1]);
                    unpack2(mul2(pack2(__bfloat162float(v[32 * i + 64]), __bfloat162float(v[32 * i + 96])), beta.y), x[i + 2], x[i + 3]);
                }
                if (!wait_warp(KS_FULL, ph)) return TURNS * c + 1;
                tc_fence_after();
                uint32_t z[16], hi[8], lo[8];
                tmem_ld_x16(tk, z);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const ulonglong2 near = *reinterpret_cast<const ulonglong2*>(&k.minus_near[16 * quarter + 2 * e]);
#pragma unroll
                    for (int f = e; f < e + 2; ++f) {
                        unpack2(fma2(f == e ? near.x : near.y, pack2(__uint_as_float(z[2 * f]), __uint_as_float(z[2 * f + 1])),
                                     pack2(x[2 * f], x[2 * f + 1])), x[2 * f], x[2 * f + 1]);
                        split2(x[2 * f], x[2 * f + 1], hi[f], lo[f]);
                    }
                }
                tmem_st_x8(mine + T_X + 8u * quarter, hi);
                tmem_st_x8(mine + T_X + 32u + 8u * quarter, lo);
                tmem_st_wait();
                tc_fence_before();
                chain_arrive(X_READY);
                // what the parts leave of X
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    unpack2(less_bf16(less_bf16(pack2(x[2 * e], x[2 * e + 1]), hi[e]), lo[e]), x[2 * e], x[2 * e + 1]);

                if (!wait_warp(U_FULL, ph)) return TURNS * c + 2;
                tc_fence_after();
                tmem_ld_x16(tk, z);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const ulonglong2 left = *reinterpret_cast<const ulonglong2*>(&k.left[16 * quarter + 2 * e]);
#pragma unroll
                    for (int f = e; f < e + 2; ++f) {
                        const uint64_t u = add2(pack2(x[2 * f], x[2 * f + 1]), pack2(__uint_as_float(z[2 * f]), __uint_as_float(z[2 * f + 1])));
                        float p, q;
                        unpack2(u, x[2 * f], x[2 * f + 1]);
                        unpack2(mul2(f == e ? left.x : left.y, u), p, q);
                        split2(p, q, hi[f], lo[f]);
                    }
                }
                tmem_st_x8(mine + T_UP + 8u * quarter, hi);
                tmem_st_x8(mine + T_UP + 32u + 8u * quarter, lo);
                tmem_st_wait();
                tc_fence_before();
                chain_arrive(UP_READY);
#pragma unroll
                for (int e = 0; e < 8; ++e) split2(x[2 * e], x[2 * e + 1], hi[e], lo[e]);
                tmem_st_x8(tk, hi);
                tmem_st_x8(tk + 8u, lo);
                tmem_st_wait();
                tc_fence_before();
                chain_arrive(U2_READY);
            }
            return chunks > 0 && !next_state(chunks - 1, false) ? TURNS * chunks : -1;
        };
        const int lost = walk();
        const bool ok = lost < 0;
        if (!ok) {
            if (lane == 0) fail();
            chain_rest(lost, chunks);
        }
        float nothing = 0.0f;   // 0, or NaN
#pragma unroll
        for (int e = 0; e < COLS; ++e) nothing = fmaf(S[e], 0.0f, nothing);
        const uint32_t odd = __ballot_sync(0xffffffffu, ok && live && chunks > 0 && !(nothing == 0.0f));   // (without tokens S moves as it is)
        if (lane == 0) odd_rows[warp] = odd;
        chain_sync();
        if (ok && live && !row_is_odd(odd_rows, warp, lane)) last_state<DK, PIECES>(a, s, part, S, quarter, row);
        __syncwarp();
    } else if (warp < kGramWarp) {
        // ------------------------------ the output ------------------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const int quad = warp - kOutWarp, row = quad * 32 + lane;
        const bool live = row0 + row < rows;
        const uint32_t mine = tmem + ((uint32_t)(quad * 32) << 16);
        unsigned char* piece_out = nullptr;   // this thread's place in the piece's outputs
        if (PIECES && piece > 0) {
            const StateSeq whole = load_state_seq(a.s, blockIdx.y, &g_delta_chunk_error);
            const long long first = delta_piece_chunk(a.p.count, whole.t0, blockIdx.y) + (piece - 1) * delta_piece_chunks(a.p, whole.n);
            piece_out = moves ? a.p.out_move + row / 64 * (kTok * 128) + 2 * (row & 7)
                              : reinterpret_cast<unsigned char*>(a.p.out + row);
            piece_out += ((first * a.v_heads + h) * rows + row0) * (long long)(kTok * 4);
        }
        bool ok = true;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            if (!wait_warp(O_FULL, (uint32_t)c & 1u)) { ok = false; break; }
            tc_fence_after();
            const Coef& k = coefs[c % kCoefStages];
            // over the values of V, which have been used, and out of shared memory in one piece
            __nv_bfloat16* const o = reinterpret_cast<__nv_bfloat16*>(smem + C::kV + (c % kVStages) * C::kVBytes + quad * (kTok * 64)) + lane;
            const uint32_t qs = mine + ((c & 1) ? T_QS_ODD : T_QS_EVEN);
#pragma unroll 1
            for (int t = 0; t < kTok; t += 16) {
                uint32_t x[16], y[16];
                tmem_ld_x16(qs + (uint32_t)t, x);
                tmem_ld_x16(mine + T_O + (uint32_t)t, y);
                tmem_ld_wait();
                if (t == kTok - 16) {
                    tc_fence_before();
                    arrive(O_EMPTY);
                }
                if (PIECES && piece > 0) {
                    // (a row over the lanes a store: 16 bytes of a row of tokens a lane took 14 us more of 82)
                    unsigned char* const tile = piece_out + (long long)c * a.v_heads * rows * (kTok * 4);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(&k.near_q[t + i]);
                        const float m[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[i + e] = __float_as_uint(fmaf(m[e], __uint_as_float(x[i + e]), __uint_as_float(y[i + e])));
                    }
                    if (!live) {
                    } else if (moves) {
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            uint32_t hi, lo;
                            split2(__uint_as_float(x[i]), __uint_as_float(x[i + 1]), hi, lo);
                            unsigned char* to = tile + (t + i) * 128;
                            const int u0 = (row % 64 / 8 ^ (i & 7)) << 4, u1 = ((row % 64 / 8 ^ (i & 7) ^ 1) << 4) + 128;
                            *reinterpret_cast<unsigned short*>(to + u0) = (unsigned short)hi;
                            *reinterpret_cast<unsigned short*>(to + u1) = (unsigned short)(hi >> 16);
                            *reinterpret_cast<unsigned short*>(to + u0 + DK * 128) = (unsigned short)lo;
                            *reinterpret_cast<unsigned short*>(to + u1 + DK * 128) = (unsigned short)(lo >> 16);
                        }
                    } else {
                        const int width = min(kRows, rows - row0);
                        float* to = reinterpret_cast<float*>(tile) + t * width;
#pragma unroll
                        for (int i = 0; i < 16; ++i) to[i * width] = __uint_as_float(x[i]);
                    }
                    __syncwarp();
                    continue;
                }
#pragma unroll
                for (int i = 0; i < 16; i += 4) {   // (all read before anything is stored)
                    const float4 f = *reinterpret_cast<const float4*>(&k.near_q[t + i]);
                    float p, q;
                    unpack2(fma2(pack2(f.x, f.y), pack2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                                 pack2(__uint_as_float(y[i]), __uint_as_float(y[i + 1]))), p, q);
                    x[i] = pack_bf16(p, q);
                    unpack2(fma2(pack2(f.z, f.w), pack2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])),
                                 pack2(__uint_as_float(y[i + 2]), __uint_as_float(y[i + 3]))), p, q);
                    x[i + 2] = pack_bf16(p, q);
                }
                const uint32_t to = smem_u32(o + 32 * t);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + 64u * i), "h"((unsigned short)x[i]) : "memory");
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + 64u * i + 64u), "h"((unsigned short)(x[i] >> 16)) : "memory");
                }
            }
            const int first = c * kTok, n = s.n - first;
            if (PIECES && piece > 0) {
                arrive(V_EMPTY + c % kVStages);
            } else if (n >= kTok) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (live) {
                        tma_store_3d(&tmap_out, smem_u32(o), row0 + row, h, s.t0 + first);
                        bulk_commit();
                        bulk_wait_read();
                    }
                    mbar_arrive(bar(V_EMPTY + c % kVStages));
                }
            } else if (live) {   // the sequence ends in this chunk
                const long long step = (long long)a.v_heads * a.dv;
                __nv_bfloat16* to = a.out + (s.t0 + first) * step + (long long)h * a.dv + row0 + row;
#pragma unroll 1
                for (int i = 0; i < n; ++i) to[i * step] = o[32 * i];
            }
            arrive(COEF_EMPTY + c % kCoefStages);
        }
        if (lane == 0) {
            bulk_wait();
            if (!ok) fail();
        }
        __syncwarp();
    } else if (warp < kInvWarp) {
        // ------------------------------ A and P from the Gram matrices ------------------------------
        // a thread a row: two warps have K K^T, two Q K^T
        const int me = warp - kGramWarp, part = me & 1, i = 32 * part + lane;
        const bool low = lane < 16, is_k = me < 2;
        const uint32_t gram = tmem + ((uint32_t)(me * 32) << 16) + T_GRAM;
        // 16 values as bf16 and what that leaves of them: two units of a row each, the second at ^ 16
        auto put16 = [&](uint32_t at, uint32_t rest, const float* z) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split2(z[8 * u + 2 * e], z[8 * u + 2 * e + 1], hi[e], lo[e]);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ 16u * u), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(rest ^ 16u * u), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
            }
        };
        // columns 8 `unit` on of this row of P; the rest of them at ^ 64
        auto p_at = [&](uint32_t P, int unit) {
            return unit < 4 ? tile_at(P, i, unit) : tile_at(P + kPRight, i - 32, unit - 4);
        };
        bool ok = true;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            Coef& k = coefs[c % kCoefStages];
            const uint32_t P = sbase + (uint32_t)(C::kTp + (c & 1) * C::kTpBytes) + 2 * kTile;
            const uint32_t A = sbase + (uint32_t)(C::kA + (c & 1) * C::kABytes);
            if (!wait_warp(COEF_FULL + c % kCoefStages, full(c, kCoefStages)) || !wait_warp(GRAM_FULL, (uint32_t)c & 1u)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t x[32];
            tmem_ld_x32(gram + 32u * part, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = low ? x[e] : x[16 + e];   // this row's own 16 columns
            float mul = k.scale_q[i];
            if (is_k) {   // K's lengths stand on the diagonal
                float kk = 0.0f;
#pragma unroll
                for (int e = 0; e < 16; ++e) kk = e == (lane & 15) ? __uint_as_float(x[e]) : kk;
                const float ik = a.norm ? rsqrtf(kk + kDeltaNormEps) : 1.0f, beta = k.beta[i];
                k.Gk[i] = make_float2(k.G[i].x, k.G[i].y - __log2f(ik));
                k.left[i] *= ik;
                k.to_end[i] *= ik;
                k.minus_near[i] = -beta * k.near[i] * ik;
                mul = beta * ik;
            } else {
                k.near_q[i] = mul * k.near[i];
            }
            arrive(LENGTHS);
            if (!wait_warp(LENGTHS, (uint32_t)c & 1u) || !wait_warp(A_EMPTY + (c & 1), free(c, kAStages)) ||
                !wait_warp(TP_EMPTY + (c & 1), free(c, kTpStages))) {
                ok = false;
                break;
            }
            const uint64_t G = pack2(k.G[i].x, k.G[i].y);
            auto decay_to = [&](float2 g) {   // e^(G_i - g)
                float p, q;
                unpack2(add2(G, pack2(-g.x, -g.y)), p, q);
                return exp2_fast(p + q);
            };
            {   // this row's own 16: the difference itself, 0 right of the diagonal
                const int j0 = 32 * part + (lane & 16);
                float z[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float4 g = *reinterpret_cast<const float4*>(&k.Gk[j0 + e]);
                    unpack2(mul2(mul2(pack2(decay_to(make_float2(g.x, g.y)), decay_to(make_float2(g.z, g.w))),
                                      pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]))), pack2(mul, mul)), z[e], z[e + 1]);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) z[e] = e - (lane & 15) < (is_k ? 0 : 1) ? z[e] : 0.0f;
                if (is_k) {
                    float* at = reinterpret_cast<float*>(smem + C::kA + (c & 1) * C::kABytes + 2 * kATile) + (i / 16) * kDiagBlock + (lane & 15);
#pragma unroll
                    for (int e = 0; e < 16; ++e) at[e * kDiagRow] = -z[e];
                } else {
                    const uint32_t at = p_at(P, j0 / 8);
                    put16(at, at ^ 64u, z);
                }
            }
            if (is_k) arrive(DIAG_FULL + (c & 1));   // (T's diagonal blocks can be begun)
            // tokens of the 16s before: through the last token of their 16, so that no factor is above 1
#pragma unroll 1
            for (int b = 0; b <= 2 * part; ++b) {
                uint32_t y[16];
                __syncwarp();
                tmem_ld_x16(gram + 16u * b, y);
                tmem_ld_wait();
                if (b == 2 * part && low) continue;
                const float f = decay_to(k.end[b]) * mul;
                float z[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 t = *reinterpret_cast<const float2*>(&k.to_end[16 * b + e]);
                    unpack2(mul2(mul2(pack2(f, f), pack2(t.x, t.y)), pack2(__uint_as_float(y[e]), __uint_as_float(y[e + 1]))),
                            z[e], z[e + 1]);
                }
                const uint32_t at = !is_k ? p_at(P, 2 * b) : b == 2 ? a_at(A, i - 48, 0) : a_at(A, i, 2 * b);
                put16(at, is_k ? at + kATile : at ^ 64u, z);
            }
            __syncwarp();
            tc_fence_before();
            arrive(GRAM_EMPTY);
            fence_proxy_async_smem();
            arrive(A_FULL + (c & 1));
        }
        if (!ok && lane == 0) fail();
        __syncwarp();
    } else if (warp < kMmaWarp) {
        // ------------------------------ T, the inverse of I + A ------------------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const int me = warp - kInvWarp;
        const bool low = lane < 16;
        uint32_t syncs = 0;
        auto sync_warps = [&] {   // the four of them
            arrive(INVERSE);
            return wait_warp(INVERSE, syncs++ & 1u);
        };
        bool ok = true;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const uint32_t T = sbase + (uint32_t)(C::kTp + (c & 1) * C::kTpBytes);
            const uint32_t A = sbase + (uint32_t)(C::kA + (c & 1) * C::kABytes);
            if (!wait_warp(DIAG_FULL + (c & 1), full(c, kAStages)) || !wait_warp(TP_EMPTY + (c & 1), free(c, kTpStages))) {
                ok = false;
                break;
            }
            {   // the diagonal blocks, one a warp, a column a lane; the upper lanes keep the lower parts
                float t[16];
                solve16(reinterpret_cast<const float*>(smem + C::kA + (c & 1) * C::kABytes + 2 * kATile) + me * kDiagBlock, lane & 15, t);
                const int col = 16 * me + (lane & 15);
                const uint32_t to = T + (uint32_t)(16 * me * 128) + 2u * (col & 7) + (low ? 0u : kTile);
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    uint32_t hi, lo;
                    split2(t[r], t[r + 1], hi, lo);
                    const uint32_t w = low ? hi : lo;
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(tile_at(to, r, col / 8)), "h"((unsigned short)w) : "memory");
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(tile_at(to, r + 1, col / 8)), "h"((unsigned short)(w >> 16)) : "memory");
                }
            }
            if (!sync_warps() || !wait_warp(A_FULL + (c & 1), full(c, kAStages))) { ok = false; break; }
            join_blocks<1>(A, T, 32 * (me >> 1) + 16, 32 * (me >> 1), me & 1, lane);
            if (!sync_warps()) { ok = false; break; }
            join_blocks<2>(A, T, 32, 0, me, lane);
            fence_proxy_async_smem();
            arrive(TP_FULL + (c & 1));
            if (lane == 0) mbar_arrive(bar(A_EMPTY + (c & 1)));
        }
        if (!ok && lane == 0) fail();
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == kMmaWarp) {
            // ------------------------------ products ------------------------------
            constexpr uint32_t kIdesc = idesc_bf16_f32(kRows, kTok), kIdescHalf = idesc_bf16_f32(kRows, kTok / 2);
            constexpr uint32_t kIdescD = idesc_bf16_f32(kRows, DK) | kIdescBMnMajor;
            bool ok = true;
            auto need = [&](int b, uint32_t parity) { ok = ok && wait_warp(b, parity); };
            auto kq = [&](int c) { return sbase + (uint32_t)(C::kKq + (c % kKqStages) * C::kKqBytes); };
            auto step = [](int kk) { return (uint64_t)((kk / 4) * (2 * kTile >> 4) + 2 * (kk % 4)); };
            // (Loops of these kept half rolled: where every SM is busy, code is what is short, 414 -> 403 us for
            // six prompts; alone, one prompt of 2048 tokens takes 137.6 us so, 136.6 unrolled.)
            // parts of S times the rows of K or Q
            auto with_state = [&](uint32_t to, uint64_t rows) {
                constexpr int kSteps = COLS / 16;   // of a thread's columns
#pragma unroll 2
                for (int kk = 0; kk < DK / 16; ++kk)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        mma_f16_ts(to, T_S + (uint32_t)(COLS * (kk / kSteps) + 8 * (kk % kSteps) + COLS / 2 * x), rows + step(kk), kIdesc,
                                   (kk | x) ? 1u : 0u);
            };
            // (+)= 64 tokens in tensor memory times a [64][64] tile
            auto with_tile = [&](uint32_t to, uint32_t left, uint32_t tile, bool more) {
                const uint64_t d = smem_desc_k_sw128(tile);
#pragma unroll
                for (int kk = 0; kk < kTok / 16; ++kk)
                    mma_f16_ts(to, left + 8 * kk, d + 2 * kk, kIdesc, (more || kk) ? 1u : 0u);
            };
            // U times P, three products of parts: outputs of 32 tokens each (the earlier need no later U)
            auto with_p = [&](uint32_t P) {
#pragma unroll 1
                for (int part = 0; part < 3; ++part) {   // hi hi, lo hi, hi lo
                    const uint32_t left = part == 1 ? T_KS + 8u : (uint32_t)T_KS;
                    const uint64_t d = smem_desc_k_sw128(P) + (part == 2 ? 4 : 0), later = d + (32 * 128 >> 4), right = d + (kPRight >> 4);
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        mma_f16_ts(T_O, left + 16 * kk, d + 2 * kk, kIdescHalf, (part | kk) ? 1u : 0u);
                        mma_f16_ts(T_O + 32, left + 16 * kk, later + 2 * kk, kIdescHalf, (part | kk) ? 1u : 0u);
                    }
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) mma_f16_ts(T_O + 32, left + 32 + 16 * kk, right + 2 * kk, kIdescHalf, 1u);
                }
            };
            // the first two Gram matrices, then in chunk c that of c + 2
#pragma unroll 1
            for (int c = -2; c < chunks; ++c) {
                const uint32_t ph = (uint32_t)c & 1u;
                const uint32_t tp = sbase + (uint32_t)(C::kTp + (c & 1) * C::kTpBytes);
                if (c >= 0) {
                    // (Q S^T goes to where the chunk before the last had its own, whose output had been read
                    // before the last chunk's P U; that has to be done with U's parts)
                    need(KQ_FULL + c % kKqStages, full(c, kKqStages));
                    if (c > 0) need(O_FULL, ph ^ 1u);
                    chain_wait(S_READY);
                    tc_fence_after();
                    if (ok && elect_one()) {
                        // (K first, for which the chain waits; both as one product of N = 128 take less of the
                        // tensor pipe, which is not what bounds this, but hold the chain for 600 clocks more)
                        with_state(T_KS, smem_desc_k_sw128(kq(c)));
                        mma_commit(bar(KS_FULL));
                        with_state((c & 1) ? T_QS_ODD : T_QS_EVEN, smem_desc_k_sw128(kq(c) + kTile));
                    }
                    __syncwarp();
                    need(TP_FULL + (c & 1), full(c, kTpStages));
                    chain_wait(X_READY);
                    tc_fence_after();
                    if (ok && elect_one()) {
                        with_tile(T_KS, T_X, tp, false);
                        with_tile(T_KS, T_X + 32, tp, true);
                        with_tile(T_KS, T_X, tp + kTile, true);
                        mma_commit(bar(U_FULL));
                    }
                    __syncwarp();
                }
                const int next = c + 2;
                if (next < chunks) {
                    need(KQ_FULL + next % kKqStages, full(next, kKqStages));
                    need(GRAM_EMPTY, ph ^ 1u);
                    tc_fence_after();
                    if (ok && elect_one()) {
                        const uint64_t d = smem_desc_k_sw128(kq(next));
#pragma unroll 4
                        for (int kk = 0; kk < DK / 16; ++kk) mma_f16_ss(T_GRAM, d + step(kk), d + step(kk), kIdesc, kk > 0);
                        mma_commit(bar(GRAM_FULL));
                    }
                    __syncwarp();
                }
                if (c >= 0) {
                    chain_wait(UP_READY);
                    tc_fence_after();
                    if (ok && elect_one()) {
                        const uint64_t d = smem_desc_mn_sw128(kq(c), 2 * kTile);
#pragma unroll
                        for (int kk = 0; kk < kTok / 16; ++kk)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                mma_f16_ts(T_S, T_UP + 8u * kk + 32u * x, d + (uint64_t)(kk * (2048 >> 4)), kIdescD, (kk | x) ? 1u : 0u);
                        mma_commit(bar(D_FULL));
                        mma_commit(bar(KQ_EMPTY + c % kKqStages));
                    }
                    __syncwarp();
                    if (c > 0) need(O_EMPTY, ph ^ 1u);
                    chain_wait(U2_READY);
                    tc_fence_after();
                    if (ok && elect_one()) {
                        with_p(tp + 2 * kTile);
                        mma_commit(bar(TP_EMPTY + (c & 1)));
                        mma_commit(bar(O_FULL));   // (of the last chunk the last: the CTA ends after it)
                    }
                    __syncwarp();
                }
            }
            if (!ok && lane == 0) fail();
            if (elect_one()) {   // what has been issued ends before the CTA does, whichever role gave up
                mma_commit(bar(DRAIN));
                (void)mbar_wait_drain(bar(DRAIN), 0u, 100000000ull);
            }
            __syncwarp();
        } else if (warp == kTmaWarp) {
            // ------------------------------ copies ------------------------------
            // V comes a chunk behind K and Q, which are wanted two chunks ahead
            const int v_tiles = min(4, (a.dv - row0 + 31) / 32);
            const uint32_t kq_bytes = (uint32_t)C::kKqBytes, v_bytes = (uint32_t)(v_tiles * kTok * 64);
            // rows past the sequence's end count as 0
            auto zero = [&](unsigned char* rows, int from, int row_bytes) {
#pragma unroll 1
                for (int i = from * (row_bytes / 16) + lane; i < kTok * (row_bytes / 16); i += 32)
                    *reinterpret_cast<uint4*>(rows + i * 16) = make_uint4(0, 0, 0, 0);
            };
            bool ok = true;
            int kqs = 0, vs = 0;   // copies begun
#pragma unroll 1
            for (int c = 0; c <= chunks && ok; ++c) {
                if (c < chunks) {
                    const int st = c % kKqStages, left = s.n - c * kTok;
                    if (!wait_warp(KQ_EMPTY + st, free(c, kKqStages))) { ok = false; break; }
                    const uint32_t at = sbase + (uint32_t)(C::kKq + st * C::kKqBytes), to = left < kTok ? bar(TAIL) : bar(KQ_FULL + st);
                    if (lane == 0) {
                        mbar_arrive_expect_tx(to, kq_bytes);
                        for (int x = 0; x < NC; ++x) {
                            tma_load_2d(at + 2 * x * kTile, &tmap_k, hk * DK + 64 * x, s.t0 + c * kTok, to);
                            tma_load_2d(at + (2 * x + 1) * kTile, &tmap_q, hk * DK + 64 * x, s.t0 + c * kTok, to);
                        }
                    }
                    ++kqs;
                    __syncwarp();
                    if (left < kTok) {
                        if (!wait_warp(TAIL, 0u)) { ok = false; break; }
#pragma unroll 1
                        for (int x = 0; x < NC; ++x) zero(smem + C::kKq + st * C::kKqBytes + 2 * x * kTile, left, 128);
                        fence_proxy_async_smem();
                        arrive(KQ_FULL + st);
                    }
                }
                if (c > 0) {
                    const int b = c - 1, st = b % kVStages, left = s.n - b * kTok;
                    if (!wait_warp(V_EMPTY + st, free(b, kVStages))) { ok = false; break; }
                    if (moves) {   // no v (and nothing else is put in its place)
                        if (b < kVStages) {
#pragma unroll 1
                            for (int x = 0; x < 4; ++x) zero(smem + C::kV + st * C::kVBytes + x * kTok * 64, 0, 64);
                        }
                        arrive(V_FULL + st);
                        continue;
                    }
                    const uint32_t at = sbase + (uint32_t)(C::kV + st * C::kVBytes), to = left < kTok ? bar(TAIL) : bar(V_FULL + st);
                    if (lane == 0) {
                        mbar_arrive_expect_tx(to, v_bytes);
#pragma unroll 1
                        for (int x = 0; x < v_tiles; ++x)
                            tma_load_2d(at + (uint32_t)(x * kTok * 64), &tmap_v, h * a.dv + row0 + 32 * x, s.t0 + b * kTok, to);
                    }
                    ++vs;
                    __syncwarp();
                    if (left < kTok) {
                        if (!wait_warp(TAIL, 1u)) { ok = false; break; }
#pragma unroll 1
                        for (int x = 0; x < v_tiles; ++x) zero(smem + C::kV + st * C::kVBytes + x * kTok * 64, left, 64);
                        fence_proxy_async_smem();
                        arrive(V_FULL + st);
                    }
                }
            }
            if (lane == 0) {
                // copies in flight land before the CTA goes away, whichever role gave up (those of the
                // sequence's end have been waited for here)
                if (!ok) fail();
                const bool tail = s.n % kTok != 0;
                auto drain = [&](int begun, int stages, int first, uint32_t parity) {
#pragma unroll 1
                    for (int i = max(0, begun - stages); i < begun; ++i) {
                        if (!tail || i < chunks - 1) (void)mbar_wait_drain(bar(first + i % stages), full(i, stages), 20000000ull);
                        else if (!ok) (void)mbar_wait_drain(bar(TAIL), parity, 20000000ull);
                    }
                };
                drain(kqs, kKqStages, KQ_FULL, 0u);
                drain(vs, kVStages, V_FULL, 1u);
            }
            __syncwarp();
        } else {
            // ------------------------------ decays, steps, lengths of q ------------------------------
            // one warp has the decays and steps of all 64 tokens, lane's and lane + 32's, their loads a chunk ahead,
            // the other the lengths of q
            const bool decays = warp == kCoefWarp;
            const DeltaHead head = delta_head(a, h);
            float2 raw[2] = {};
            auto load = [&](int c) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int t = c * kTok + 32 * x + lane;
                    if (t < s.n) raw[x] = delta_raw_gates(a, s.t0 + t, h);
                }
            };
            if (decays && chunks > 0) load(0);
            bool ok = true;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const int ks = c % kKqStages, cs = c % kCoefStages;
                Coef& k = coefs[cs];
                if (!wait_warp(COEF_EMPTY + cs, free(c, kCoefStages))) { ok = false; break; }
                if (decays) {
                    // the running sums, in 64 bits of which 40 stand behind the point
                    long long G[2], all = 0;
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) {
                        const int i = 32 * x + lane;
                        const float2 in = x ? raw[1] : raw[0];
                        const float2 gate = c * kTok + i < s.n ? delta_gates(head, in) : make_float2(0.0f, 0.0f);
                        k.beta[i] = fmaf(gate.x, 0.0f, gate.y);   // (a decay that is no number makes the step none)
                        long long sum = fixed_log2(gate.x);
#pragma unroll 1
                        for (int o = 1; o < 32; o <<= 1) {
                            const long long y = __shfl_up_sync(0xffffffffu, sum, o);
                            if (lane >= o) sum += y;
                        }
                        sum += all;
                        all = __shfl_sync(0xffffffffu, sum, 31);
                        if (x) G[1] = sum;
                        else G[0] = sum;
                    }
                    if (c + 1 < chunks) load(c + 1);
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) {
                        const int i = 32 * x + lane;
                        const long long sum = x ? G[1] : G[0], end = __shfl_sync(0xffffffffu, sum, lane | 15);
                        const float hi = unfixed(sum);
                        const float2 both = make_float2(hi, unfixed(sum - __float2ll_rn(hi * 1099511627776.0f)));
                        k.near[i] = exp2_fast(hi);
                        k.left[i] = exp2_fast(unfixed(all - sum));
                        k.to_end[i] = exp2_fast(unfixed(end - sum));
                        k.G[i] = both;
                        if ((lane & 15) == 15) k.end[i / 16] = both;
                    }
                    if (lane == 0) k.last = exp2_fast(unfixed(all));
                } else {
                    if (!wait_warp(KQ_FULL + ks, full(c, kKqStages))) { ok = false; break; }
#pragma unroll 1
                    for (int i = lane; i < kTok; i += 32) {
                        float iq = 1.0f;
                        if (a.norm) {
                            const unsigned char* at = smem + C::kKq + ks * C::kKqBytes + (kTok + i) * 128;
                            uint64_t q2 = 0, r2 = 0;
#pragma unroll 1
                            for (int x = 0; x < NC; ++x, at += 2 * kTile)
#pragma unroll 2
                                for (int u = 0; u < 8; ++u) {
                                    const uint4 w = *reinterpret_cast<const uint4*>(at + ((u ^ (i & 7)) << 4));
                                    auto two = [](uint32_t v) { return pack2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u)); };
                                    const uint64_t w0 = two(w.x), w1 = two(w.y), w2 = two(w.z), w3 = two(w.w);
                                    q2 = fma2(w0, w0, q2);
                                    r2 = fma2(w1, w1, r2);
                                    q2 = fma2(w2, w2, q2);
                                    r2 = fma2(w3, w3, r2);
                                }
                            float x, y;
                            unpack2(add2(q2, r2), x, y);
                            iq = rsqrtf(x + y + kDeltaNormEps);
                        }
                        k.scale_q[i] = a.scale * iq;
                    }
                }
                arrive(COEF_FULL + cs);
            }
            if (!ok && lane == 0) fail();
            __syncwarp();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    uint32_t any_odd = 0;
#pragma unroll 1
    for (int i = 0; i < kOutWarp; ++i) any_odd |= odd_rows[i];
    if (any_odd && warp < kOutWarp) redo<DK, PIECES>(a, s, part, odd_rows, smem);
}

// [T][heads * dim] as the TMA sees it, a box of `box` values of 64 tokens.
bool make_token_map(CUtensorMap* m, const __nv_bfloat16* base, long long stride, int width, int T, int box_width) {
    auto enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dim[2] = {(cuuint64_t)width, (cuuint64_t)T};
    const cuuint64_t step[1] = {(cuuint64_t)(stride > width ? stride : width) * 2};   // (one token: any stride)
    const cuuint32_t box[2] = {(cuuint32_t)box_width, kTok};
    const cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<__nv_bfloat16*>(base), dim, step, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, box_width == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The output, [T][heads][dv]: a box of 32 values of one head and 64 tokens; what
// lies past a head's last value is not written.
bool make_out_map(CUtensorMap* m, __nv_bfloat16* base, int heads, int dv, int T) {
    auto enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dim[3] = {(cuuint64_t)dv, (cuuint64_t)heads, (cuuint64_t)T};
    const cuuint64_t step[2] = {(cuuint64_t)dv * 2, (cuuint64_t)dv * heads * 2};
    const cuuint32_t box[3] = {32, 1, kTok};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dim, step, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int DK>
cudaError_t launch(const DeltaArgs& a, cudaStream_t stream) {
    using C = Cfg<DK>;
    CUtensorMap mq, mk, mv, mo;
    if (!make_token_map(&mq, a.q, a.q_token, a.k_heads * DK, a.s.T, 64) ||
        !make_token_map(&mk, a.k, a.k_token, a.k_heads * DK, a.s.T, 64) ||
        !make_token_map(&mv, a.v, a.v_token, a.v_heads * a.dv, a.s.T, 32) || !make_out_map(&mo, a.out, a.v_heads, a.dv, a.s.T))
        return cudaErrorInvalidValue;
    auto kernel = a.p.count > 1 ? delta_chunk_kernel<DK, true> : delta_chunk_kernel<DK, false>;
    static bool attr_set[64][2] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev][a.p.count > 1]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev][a.p.count > 1] = true;
    }
    return launch_pdl(kernel, dim3((unsigned)((a.dv + kRows - 1) / kRows * a.v_heads), (unsigned)a.s.B, (unsigned)(2 * a.p.count - 1)),
                      dim3(kThreads), C::kSmem, stream, true, mq, mk, mv, mo, a);
}

// The chain and the issuing warp over six chunks, from the third of which on nothing comes after a
// turn: the chain's waits run out while the issuing warp still is in a longer one of its own.
__global__ void __launch_bounds__(kChainThreads) delta_wait_selftest_kernel(uint32_t tries) {
    __shared__ __align__(8) uint64_t bars[4];
    enum { KS, U, D, NEVER };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(bar(i), 1);
        fence_barrier_init();
    }
    __syncthreads();
    constexpr int kChunks = 6;
    bool ok = true;
    if (warp < kOutWarp) {
        auto walk = [&] {
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                const uint32_t ph = (uint32_t)c & 1u;
                if (c > 0 && !wait_warp(bar(D), ph ^ 1u, tries)) return TURNS * c;
                chain_arrive(S_READY);
                if (!wait_warp(bar(KS), ph, tries)) return TURNS * c + 1;
                chain_arrive(X_READY);
                if (!wait_warp(bar(U), ph, tries)) return TURNS * c + 2;
                chain_arrive(UP_READY);
                chain_arrive(U2_READY);
            }
            return -1;
        };
        const int lost = walk();
        ok = lost < 0;
        if (!ok) chain_rest(lost, kChunks);
    } else {
        auto done = [&](int b) {
            if (ok && lane == 0) mbar_arrive(bar(b));
        };
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
            if (c == 2) ok = wait_warp(bar(NEVER), 0u, 4 * tries);
            chain_wait(S_READY);
            done(KS);
            chain_wait(X_READY);
            done(U);
            chain_wait(UP_READY);
            done(D);
            chain_wait(U2_READY);
        }
    }
    if (!ok && lane == 0) report_device_error(&g_delta_chunk_error, TERN_DEVERR_DELTA_WAIT);
}

}  // namespace

cudaError_t launch_delta_wait_selftest(uint64_t limit_ns, cudaStream_t stream) {
    const uint64_t tries = limit_ns / kWaitNap;
    delta_wait_selftest_kernel<<<1, kChainThreads, 0, stream>>>(tries > 0 ? (uint32_t)tries : 1u);
    return cudaGetLastError();
}

cudaError_t launch_delta_chunk(const DeltaArgs& a, cudaStream_t stream) {
    return a.dk == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

cudaError_t read_delta_chunk_device_error(int* code) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_delta_chunk_error, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_delta_chunk_error, &zero, sizeof(int));
}

}  // namespace tern
