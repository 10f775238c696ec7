// Attention over whole prompts (packed sequences, grouped heads, causal) on
// the fifth-generation tensor cores.
//
//   S = Q K^T      M = 128 rows, N = 128 keys, K = head dim   (kind::f16)
//   P = 2^(c S - c m), c = softmax_scale * log2 e, m the row's reference maximum
//   O += P V       M = 128 rows, N = head dim, K = 128 keys, P from tensor memory
//
// Rows.  A row is a (query token, query head of the group) pair, token-major:
// a tile of 128 rows covers 128 / G tokens (rounded down) of one kv head, so
// grouped heads share every K and V tile and a short prompt fills a tile G
// times sooner.  One tensor copy with the box {64 channels, G heads, 128 / G
// tokens} lands them in that order.
//
// Up to head dim 128 a CTA carries two such tiles (consecutive tokens) over
// the same K and V blocks: the tensor pipe works on one tile's products while
// the other tile's softmax runs on its own warpgroup.  At head dim 256 the
// output accumulator takes half of tensor memory, so one tile is carried with
// two buffers of S; the two warpgroups take 64 of its 128 columns each and
// agree on the row maximum through shared memory.
//
// Softmax in the exp2 domain, one thread per row (tensor-memory lane), with a
// lazy maximum: the reference m moves only when a score passes it by more
// than 2^8 (P then stays at most 2^8, which f16 and bf16 hold with full
// relative precision); only then is O rescaled, by the softmax warps
// themselves.  Row sums use the unrounded weights.
//
// Persistent CTAs, one per SM, take the tiles longest first, in rounds of
// alternating direction, so that every CTA gets about the same work without a
// counter in memory.  The i-th longest tile is found by one warp, ahead of its
// use, by counting for a bisected number of key blocks c how many tiles visit
// at least c blocks (a closed form per sequence): no plan kernel, no workspace.
// Copies of the next tile's Q, K and V and its first S run under the end of the
// current tile.
//
// What bounds it.  A block of 128 keys costs a CTA 2048 cycles of the tensor
// pipe (two row tiles, or one of head dim 256), and at head dim 128 the operands
// of S alone read shared memory at its full 128 bytes a cycle, beside the copies.
// Measured on a GB300: one 16384-token prompt, 32 / 8 heads, head dim 128, bf16
// 1.43 ms = 1.53 PFLOP/s of the visible pairs (0.80 of the measured bf16 rate,
// about 2700 cycles a block); head dim 256, four prompts of 1024-4096 tokens
// 0.47 ms = 1.31 PFLOP/s (0.68; copies, S and P.V together ask 2500 cycles a block
// of shared memory).  What was tried: one row tile per CTA and no persistent loop
// (1.68 ms), the MMAs issued from a single-lane branch (1.90 ms).
//
// Masked keys.  Their scores are replaced by -inf, so P is exactly 0 there; but
// 0 * NaN is NaN, so their V rows must not meet the product when they hold
// infinities or NaN.  V rows past the sequence are zeroed in shared memory.  V
// rows of the same sequence that some row of the tile does not see (the blocks
// on the diagonal) are looked over by one warp; where it finds a value that
// is not finite, the tile's outputs are summed again, row by row over the
// visible keys alone, from the maxima and sums already known.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "pa_attn.cuh"
#include "pa_tc_warp.cuh"

namespace pa {

struct PromptParams {
    const int32_t *cu_q;
    const int32_t *cu_k;
    void *out;
    float *lse;
    uint32_t *dev_error;
    int B, total_q, total_k, Hq, Hkv, G;
    int tpt;     // query tokens per 128-row tile: 128 / G
    int max_tiles;    // of one kv head, for ascending prefix sums
    unsigned tq_mul;  // floor(2^32 / query tokens per CTA tile) + 1
    int out_dtype, causal;
    const uint16_t *q, *k, *v;  // (for the rows summed again)
    long long qs, ks, vs;       // elements between rows
    float softmax_scale;
};

namespace prompt {

using namespace tc;

constexpr int BN = 128;                 // keys per block
constexpr float SLACK = 8.0f;           // exp2-domain headroom of the lazy maximum
constexpr int W_LOAD = 8, W_MMA = 9, W_SCHED = 10, W_LOOK = 11;  // warps 0-3, 4-7: softmax
constexpr int THREADS = 384;            // (the third warpgroup gives registers to the softmax)
constexpr int NINFO = 4;                // tiles announced ahead
// registers per thread after the split: 168 at launch (384 x 168 = 256 x 216 + 128 x 72)
constexpr int REGS_LAUNCH = 168, REGS_SOFTMAX = 216, REGS_OTHER = 72;
static_assert(256 * REGS_SOFTMAX + 128 * REGS_OTHER <= THREADS * REGS_LAUNCH, "register split exceeds the launch");

template <int D>
struct Lay {
    static constexpr bool DUAL = D <= 128;           // two row tiles, or one with two S buffers
    static constexpr int QT = DUAL ? 2 : 1;
    static constexpr int NCOL = DUAL ? 128 : 64;     // S columns per softmax thread
    static constexpr int PANELS = D / 64;            // 128-byte panels of a row
    static constexpr int TILE = BN * D * 2;          // one K or V tile
    static constexpr int NU = D == 256 ? 2 : 1;      // ring units per tile
    static constexpr int UNIT = TILE / NU;
    static constexpr int NS = D == 64 ? 12 : 5;      // ring units
    static constexpr int Q_BYTES = 128 * D * 2;
    static constexpr int Q_OFF = 0;
    static constexpr int KV_OFF = QT * Q_BYTES;
    static constexpr int RED_OFF = KV_OFF + NS * UNIT;   // [2 buffers][2 halves][128] floats (D = 256: maxima, sums)
    static constexpr int BAR_OFF = RED_OFF + (DUAL ? 0 : 4 * 128 * 4);
    enum {
        B_Q = 0,                 // [2] query tile landed
        B_QFREE = B_Q + 2,       // [2] its last S complete
        B_FULL = B_QFREE + 2,    // [NS]
        B_FREE = B_FULL + NS,    // [NS]
        B_S = B_FREE + NS,       // [2] S complete (per row tile, or per buffer)
        B_P = B_S + 2,           // [2] P written, O rescaled
        B_O = B_P + 2,           // [2] dual: the tile's last P.V complete; else [0] every P.V
        B_OFREE = B_O + 2,       // [2] O read out
        B_INFO = B_OFREE + 2,    // [NINFO] a tile announced
        B_INFOFREE = B_INFO + NINFO,
        B_LOOK = B_INFOFREE + NINFO,  // [NINFO] the tile's V rows looked over
        B_WG = B_LOOK + NINFO,  // the eight softmax warps (D = 256)
        B_EXIT = B_WG + 1,          // the softmax warps have left
        B_DONE = B_EXIT + 1,
        NBARS = B_DONE + 1
    };
    static constexpr int INFO_OFF = (BAR_OFF + NBARS * 8 + 15) / 16 * 16;  // [NINFO] 8 words
    static constexpr int MISC_OFF = INFO_OFF + NINFO * 32;                 // [0] tmem, [1] abort, [2] errors
    static constexpr int SMEM = MISC_OFF + 16;
    static constexpr int TM_O = 256, TM_COLS = 512;
    static_assert(SMEM <= 227 * 1024, "prompt kernel exceeds the shared memory of one CTA");
};

struct Seq {
    int nt;              // tiles
    int q0, lq, k0, lk;  // lk < 0: the key range breaks the contract; lq = 0 when the query range does
    bool bad;
};

__device__ __forceinline__ int per_tile(const PromptParams &P, int x, int tq);

__device__ __forceinline__ Seq load_seq(const PromptParams &P, int s, int tq) {
    Seq r;
    const int a = P.cu_q[s], b = P.cu_q[s + 1], c = P.cu_k[s], d = P.cu_k[s + 1];
    const bool okq = a >= 0 && a <= b && b <= P.total_q, okk = c >= 0 && c <= d && d <= P.total_k;
    r.q0 = a;
    r.lq = okq ? b - a : 0;
    r.k0 = c;
    r.lk = okk ? d - c : -1;
    r.nt = per_tile(P, r.lq + tq - 1, tq);
    r.bad = !okq || !okk;
    return r;
}

// x / tq: the high word of a product where that is exact (x * tq < 2^32)
__device__ __forceinline__ int per_tile(const PromptParams &P, int x, int tq) {
    return tq > 1 && x < (1 << 24) ? (int)__umulhi((unsigned)x, P.tq_mul) : x / tq;
}

// tiles of `tq` query tokens that visit at least c blocks of keys: the last
// `count` of the sequence's nt tiles (blocks grow with the tile)
__device__ __forceinline__ int tiles_with(const PromptParams &P, int lq, int lk, int nt, int c, int tq) {
    if (c <= 0) return nt;
    const int need = (c - 1) * BN;  // visible keys of the tile's last row must exceed this
    if (lk <= need) return 0;
    if (!P.causal) return nt;
    const int x = need - (lk - lq);
    const int first = x < 0 ? 0 : min(per_tile(P, x, tq), nt - 1);
    return nt - first;
}

// A tile as its roles see it
struct Tile {
    int seq, tile, g;      // seq < 0: no more tiles
    int q0, lq, k0, lk;    // packed rows of the sequence; lk < 0: its key range breaks the contract
};

// The want-th tile, longest first, by one whole warp.  `first` holds the two
// sequences (lane, lane + 32) of this lane.
struct Search {
    Seq first[2];
    int tiles;               // of one kv head
    // where the last tile was found: its number of blocks, the tiles with more and
    // with as many, the 32 sequences it is among and the tiles of that class before
    // them.  Tiles are asked for in order, so most are found from here: every CTA
    // looks through the sequences a few times per number of blocks, not per tile.
    int top, above, cnt, base, before;
};

__device__ __forceinline__ void restart(Search &S, int top) {
    S.top = top;
    S.above = S.cnt = S.base = S.before = 0;
}

template <typename F>
__device__ __forceinline__ int over_seqs(const PromptParams &P, const Search &S, int TQ, F &&f) {
    const int lane = threadIdx.x & 31;
    int n = 0;
#pragma unroll 4
    for (int s = lane, i = 0; s < P.B; s += 32, ++i) n += f(i == 0 ? S.first[0] : i == 1 ? S.first[1] : load_seq(P, s, TQ));
    return __reduce_add_sync(0xffffffffu, n);
}

__device__ __forceinline__ Tile find_tile(const PromptParams &P, Search &S, int TQ, unsigned idx) {
    const int lane = threadIdx.x & 31;
    Tile t;
    t.seq = -1;
    t.tile = t.q0 = t.lq = t.k0 = t.lk = 0;
    const unsigned w = idx / (unsigned)P.Hkv;  // (tiles of all kv heads are counted in 31 bits, and one round more fits)
    t.g = (int)(idx - w * (unsigned)P.Hkv);
    if (w >= (unsigned)S.tiles) return t;
    const int want = (int)w;
    // (all tiles in one round of the CTAs: their order does not matter)
    const bool one_round = (unsigned)S.tiles * (unsigned)P.Hkv <= gridDim.x;
    if (one_round) S.cnt = S.tiles;
    if (want >= S.cnt) {
        // another class: count(lo) > want >= count(hi); tiles come longest first, so a
        // later one has at most the blocks of the one before
        int lo = 0, hi = S.top + 1;
        S.cnt = S.tiles;
        S.above = over_seqs(P, S, TQ, [&](const Seq &q) { return tiles_with(P, q.lq, q.lk, q.nt, hi, TQ); });
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            const int n = over_seqs(P, S, TQ, [&](const Seq &q) { return tiles_with(P, q.lq, q.lk, q.nt, mid, TQ); });
            if (n > want) {
                lo = mid;
                S.cnt = n;
            } else {
                hi = mid;
                S.above = n;
            }
        }
        S.top = lo;
        S.base = S.before = 0;
    }
    // the (want - above)-th, by sequence, of the tiles with exactly `top` blocks
    const int rank = want - S.above, lo = S.top;
    int before = S.before;
    for (int base = S.base; base < P.B; base += 32) {
        const int i = base >> 5;
        const int s = base + lane;
        Seq q;
        q.lq = q.nt = 0;
        int n = 0, from = 0;
        if (s < P.B) {
            q = i == 0 ? S.first[0] : i == 1 ? S.first[1] : load_seq(P, s, TQ);
            n = q.nt;
            if (!one_round) {
                const int ge = tiles_with(P, q.lq, q.lk, q.nt, lo, TQ);
                n = ge - tiles_with(P, q.lq, q.lk, q.nt, lo + 1, TQ);
                from = q.nt - ge;
            }
        }
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        const int ex = before + x - n;
        const unsigned mine = __ballot_sync(0xffffffffu, rank >= ex && rank < ex + n);
        if (mine) {
            const int from_lane = __ffs(mine) - 1;
            S.base = base;
            S.before = before;
            t.seq = base + from_lane;
            t.tile = __shfl_sync(0xffffffffu, from + rank - ex, from_lane);
            t.q0 = __shfl_sync(0xffffffffu, q.q0, from_lane);
            t.lq = __shfl_sync(0xffffffffu, q.lq, from_lane);
            t.k0 = __shfl_sync(0xffffffffu, q.k0, from_lane);
            t.lk = __shfl_sync(0xffffffffu, q.lk, from_lane);
            return t;
        }
        before += __shfl_sync(0xffffffffu, x, 31);
    }
    return t;
}

// position in the order of tiles of this CTA's r-th one: rounds of alternating direction
__device__ __forceinline__ unsigned nth_tile(int r) {
    return (unsigned)r * gridDim.x + ((r & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS, 1)
    pa_prompt_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv, PromptParams P) {
    using Y = Lay<D>;
    constexpr bool DUAL = Y::DUAL;
    constexpr int NS = Y::NS, NU = Y::NU, QT = Y::QT;
    // (the kernel has no static shared memory, so the dynamic part starts on its
    // declared alignment; the swizzled tiles depend on it, hence the check)
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    if (sb & 1023) {
        if (threadIdx.x == 0 && P.dev_error) atomicOr(P.dev_error, PA_DEV_ERR_TIMEOUT);
        return;
    }
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Y::BAR_OFF);
    int *misc = reinterpret_cast<int *>(smem + Y::MISC_OFF);
    volatile int *abort = misc + 1;
    float *red = reinterpret_cast<float *>(smem + Y::RED_OFF);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const float NaN = __int_as_float(0x7fc00000);
    const int TQ = P.tpt * QT;

    // set up while the kernel before drains, read nothing of its writes before it has
    grid_dependents_launch();
    Search S;  // (the scheduler's: asked for before the barriers are met below)
    S.first[0].lq = S.first[0].lk = S.first[0].nt = 0;
    S.first[1] = S.first[0];
    S.tiles = 0;
    restart(S, 0);
    if (warp == W_SCHED) {
        grid_dependency_wait();
        if (lane < P.B) S.first[0] = load_seq(P, lane, TQ);
        if (lane + 32 < P.B) S.first[1] = load_seq(P, lane + 32, TQ);
    }
    if (tid < Y::NBARS) {
        const int i = tid;
        uint32_t c = 1;
        if (i >= Y::B_P && i < Y::B_P + 2) c = DUAL ? 4 : 8;
        if (i >= Y::B_OFREE && i < Y::B_OFREE + 2) c = DUAL ? 4 : 8;
        if (i >= Y::B_INFOFREE && i < Y::B_INFOFREE + NINFO) c = 11;  // load, MMA, look, eight softmax warps
        if (i >= Y::B_FREE && i < Y::B_FREE + NS) c = 2;              // MMA, look
        if (i == Y::B_WG || i == Y::B_EXIT) c = 8;
        mbar_init(&bars[i], c);
        mbar_fence_init();
    }
    if (tid == 128) {
        misc[1] = 0;
        misc[2] = 0;
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    if (warp == W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + Y::MISC_OFF),
                     "r"(Y::TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_dependency_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform(misc[0]);
    uint32_t err = 0;

    // the r-th announced tile; its entry stays until every role has freed it
    auto entry = [&](int r) -> Tile {
        const volatile int *p = reinterpret_cast<const volatile int *>(smem + Y::INFO_OFF + (r % NINFO) * 32);
        Tile t;
        t.seq = p[0];
        t.tile = p[1];
        t.g = p[2];
        t.q0 = p[3];
        t.lq = p[4];
        t.k0 = p[5];
        t.lk = p[6];
        return t;
    };
    // ... once it is announced (a whole warp, or one thread)
    auto info = [&](int r, bool one) -> Tile {
        const int i = r % NINFO;
        const bool ok = one ? sleep_wait<false>(&bars[Y::B_INFO + i], (r / NINFO) & 1, abort, err)
                            : sleep_wait(&bars[Y::B_INFO + i], (r / NINFO) & 1, abort, err);
        if (ok) return entry(r);
        Tile t;
        t.seq = -1;
        t.tile = t.g = t.q0 = t.lq = t.k0 = t.lk = 0;
        return t;
    };
    // per row tile x: first token, tokens, blocks of keys
    auto rows_of = [&](const Tile &t, int x, int &tok0, int &ntok) -> int {
        tok0 = (t.tile * QT + x) * P.tpt;
        ntok = min(P.tpt, t.lq - tok0);
        if (t.seq < 0 || ntok <= 0 || t.lk <= 0) return 0;
        const int vis = P.causal ? min(t.lk, t.lk - t.lq + tok0 + ntok) : t.lk;
        return vis > 0 ? (vis + BN - 1) / BN : 0;
    };

    // ring unit v of a tile with n blocks, in the order the products need them:
    // whether it is V's, of which block, which half (head dim 256)
    auto unit_of = [&](int v, int n, bool &isv, int &j, int &half) {
        const int q = v / NU;
        half = v % NU;
        if (DUAL) {  // K0 V0 K1 V1 ...
            isv = q & 1;
            j = q >> 1;
        } else {     // K0 K1 V0 K2 V1 ... V(n-1)
            isv = q > 0 && ((q & 1) == 0 || q == 2 * n - 1);
            j = q == 0 ? 0 : q == 2 * n - 1 ? n - 1 : isv ? q / 2 - 1 : (q + 1) / 2;
        }
    };

    if (warp >= W_LOAD) {
        regs_dec<REGS_OTHER>();  // the whole third warpgroup
        if (warp == W_SCHED) {
            // ================================================== tiles
            bool bad = false;
            int longest = 0;
            {
                int n = 0;
                for (int s = lane, i = 0; s < P.B; s += 32, ++i) {
                    const Seq q = i < 2 ? S.first[i] : load_seq(P, s, TQ);
                    bad |= q.bad;
                    n += q.nt;
                    longest = max(longest, q.lk);
                }
                S.tiles = __reduce_add_sync(0xffffffffu, n);
                longest = __reduce_max_sync(0xffffffffu, longest);
            }
            // (prefix sums that go back and forth could name the same rows many times over)
            if (S.tiles < 0 || S.tiles > P.max_tiles) {
                S.tiles = 0;
                bad = true;
            }
            if (bad && blockIdx.x == 0 && P.dev_error) atomicOr(P.dev_error, PA_DEV_ERR_CONTEXT_LEN);
            const int top0 = (longest + BN - 1) / BN;
            restart(S, top0);
            bool failed = false;  // a wait ran out: the rows of the tiles not yet written become NaN
            for (int r = 0;; ++r) {
                const Tile t = find_tile(P, S, TQ, nth_tile(r));
                if (failed) {
                    if (t.seq < 0) break;
                    for (int i = 0; i < TQ && t.tile * TQ + i < t.lq; ++i) {
                        const size_t row = (size_t)(t.q0 + t.tile * TQ + i) * P.Hq + (size_t)t.g * P.G;
                        for (int e = lane; e < P.G * D; e += 32) {
                            if (P.out_dtype == PA_F32) reinterpret_cast<float *>(P.out)[row * D + e] = NaN;
                            else reinterpret_cast<uint16_t *>(P.out)[row * D + e] = 0x7FFF;  // a NaN of f16 and of bf16
                        }
                        for (int e = lane; e < P.G && P.lse != nullptr; e += 32) P.lse[row + e] = NaN;
                    }
                    continue;
                }
                const int i = r % NINFO;
                int back = -1;  // the first tile that may be unwritten
                if (r >= NINFO && !sleep_wait(&bars[Y::B_INFOFREE + i], (r / NINFO - 1) & 1, abort, err)) {
                    back = r - NINFO;
                } else {
                    if (lane == 0) {
                        int4 *p = reinterpret_cast<int4 *>(smem + Y::INFO_OFF + i * 32);
                        p[0] = make_int4(t.seq, t.tile, t.g, t.q0);
                        p[1] = make_int4(t.lq, t.k0, t.lk, 0);
                        mbar_arrive(&bars[Y::B_INFO + i]);
                    }
                    __syncwarp();
                    if (t.seq >= 0) continue;
                    // all announced: see them through
                    for (int d = max(0, r - NINFO + 1); d < r && back < 0; ++d)
                        if (!sleep_wait(&bars[Y::B_INFOFREE + d % NINFO], (d / NINFO) & 1, abort, err)) back = d;
                    if (back < 0) break;
                }
                failed = true;
                (void)mbar_wait_bounded(&bars[Y::B_EXIT], 0, nullptr);
                __syncwarp();
                restart(S, top0);
                r = back - 1;
            }
        } else if (warp == W_LOAD) {
            // ================================================== tensor copies
            if (lane == 0) {
                const uint32_t qbytes = (uint32_t)(P.tpt * P.G) * 128u * Y::PANELS;
                int u = 0, nq[2] = {0, 0};
                bool ok = true;
#ifdef PA_FAULT_INJECT
                // the copy of ring unit (word >> 8) - 1 of CTA 0 goes missing
                const uint32_t fi = P.dev_error && blockIdx.x == 0 ? *P.dev_error >> 8 : 0u;
#endif
                for (int r = 0; ok; ++r) {
                    const Tile t = info(r, true);
                    if (t.seq < 0) break;
                    int tok0[2], ntok[2], nblk[2] = {0, 0};
#pragma unroll
                    for (int x = 0; x < QT; ++x) nblk[x] = rows_of(t, x, tok0[x], ntok[x]);
                    const int n = max(nblk[0], nblk[1]);
                    auto copy_q = [&](int x) {
                        if (nblk[x] == 0) return;
                        if (nq[x] > 0) ok = ok && sleep_wait<false>(&bars[Y::B_QFREE + x], (nq[x] - 1) & 1, abort, err);
                        if (!ok) return;
                        ++nq[x];
                        mbar_arrive_expect_tx(&bars[Y::B_Q + x], qbytes);
#pragma unroll
                        for (int c = 0; c < Y::PANELS; ++c)
                            tma_load_4d(smem + Y::Q_OFF + x * Y::Q_BYTES + c * 128 * 128, &tq, &bars[Y::B_Q + x],
                                        64 * c, 0, t.q0 + tok0[x], t.g);
                    };
                    const int units = 2 * n * NU;
                    for (int v = 0; v < units && ok; ++v, ++u) {
                        if (v == 0) copy_q(0);
                        const int slot = u % NS;
                        if (ok && u >= NS) ok = sleep_wait<false>(&bars[Y::B_FREE + slot], ((u / NS) - 1) & 1, abort, err);
                        if (!ok) break;
                        bool isv;
                        int j, half;
                        unit_of(v, n, isv, j, half);
                        uint8_t *dst = smem + Y::KV_OFF + slot * Y::UNIT;
                        const int key = t.k0 + j * BN;
#ifdef PA_FAULT_INJECT
                        if (fi != 0 && u + 1 == (int)fi) continue;
#endif
                        mbar_arrive_expect_tx(&bars[Y::B_FULL + slot], Y::UNIT);
                        if (NU == 1) {
#pragma unroll
                            for (int c = 0; c < Y::PANELS; ++c)
                                tma_load_4d(dst + c * BN * 128, isv ? &tv : &tk, &bars[Y::B_FULL + slot], 64 * c, key,
                                            t.g, 0);
                        } else if (!isv) {                     // channels 128 * half ..: two panels of 128 keys
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                tma_load_4d(dst + c * BN * 128, &tk, &bars[Y::B_FULL + slot], 128 * half + 64 * c, key,
                                            t.g, 0);
                        } else {                               // keys 64 * half ..: four panels of 64 keys
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                tma_load_4d(dst + c * 64 * 128, &tv, &bars[Y::B_FULL + slot], 64 * c, key + 64 * half,
                                            t.g, 0);
                        }
                        if (QT == 2 && v == 0) copy_q(1);
                    }
                    mbar_arrive(&bars[Y::B_INFOFREE + r % NINFO]);
                }
                if (*abort) {  // let every copy still in flight land before the CTA exits
#pragma unroll
                    for (int x = 0; x < QT; ++x)
                        if (nq[x] > 0) (void)mbar_wait_bounded(&bars[Y::B_Q + x], (nq[x] - 1) & 1, nullptr);
                    for (int i = max(0, u - NS); i < u; ++i) {
#ifdef PA_FAULT_INJECT
                        if (fi != 0 && i + 1 == (int)fi) continue;
#endif
                        (void)mbar_wait_bounded(&bars[Y::B_FULL + i % NS], (i / NS) & 1, nullptr);
                    }
                }
            }
            __syncwarp();
        } else if (warp == W_MMA) {
            // ================================================== MMA issue
            constexpr uint32_t FMT = BF16 ? (1u << 7) | (1u << 10) : 0u;
            constexpr uint32_t ID_S = idesc(128, BN, 0) | FMT;
            constexpr uint32_t ID_O = idesc(128, D, 0) | FMT | (1u << 16);  // B = V read MN-major
            // The issuing warp is on the critical path (its waits and address arithmetic
            // are not hidden by the tensor pipe's short queue): the ring
            // position is a counter, descriptors are a base plus a multiple of it.
            struct Pos {
                int slot, par;  // ring slot, parity of its phase
                __device__ __forceinline__ Pos next() const {
                    const bool wrap = slot == NS - 1;
                    Pos r;
                    r.slot = wrap ? 0 : slot + 1;
                    r.par = par ^ (wrap ? 1 : 0);
                    return r;
                }
            };
            auto full = [&](Pos p) { return sleep_wait(&bars[Y::B_FULL + p.slot], p.par, abort, err); };
            auto freed = [&](Pos p) { mma_commit_w(&bars[Y::B_FREE + p.slot]); };
            const uint64_t qd = sdesc(sb + Y::Q_OFF, 16, 1024, 2), kd = sdesc(sb + Y::KV_OFF, 16, 1024, 2),
                           vd = sdesc(sb + Y::KV_OFF, BN / NU * 128, 1024, 2);
            // S = Q K^T over one unit of K (all channels, or 128 of them)
            auto issue_qk = [&](int x, uint32_t dS, Pos p, int half) {
                const uint64_t a = qd + (uint32_t)((x * Y::Q_BYTES + half * 2 * 128 * 128) >> 4);
                const uint64_t b = kd + (uint32_t)(p.slot * (Y::UNIT >> 4));
                constexpr int STEPS = D / 16 / NU;
#pragma unroll
                for (int k = 0; k < STEPS; ++k) {
                    const uint32_t o = (uint32_t)((k >> 2) * (128 * 128) + 32 * (k & 3)) >> 4;
                    mma_f16_w(dS, a + o, b + o, ID_S, (half > 0 || k > 0) ? 1u : 0u);
                }
            };
            // O += P V over one unit of V (128 or 64 keys)
            auto issue_pv = [&](uint32_t dO, uint32_t aP, Pos p, int half, bool first) {
                constexpr int KEYS = BN / NU;
                const uint64_t b = vd + (uint32_t)(p.slot * (Y::UNIT >> 4));
#pragma unroll
                for (int k = 0; k < KEYS / 16; ++k)
                    mma_f16_ts_w(dO, aP + (uint32_t)(half * KEYS / 2 + 8 * k), b + (uint32_t)((k * 16 * 128) >> 4), ID_O,
                               (!first || half > 0 || k > 0) ? 1u : 0u);
            };
            {
                bool ok = true;
                int tok0, ntok;  // (not used here)
                Pos pos;         // of the next unit
                pos.slot = pos.par = 0;
                if constexpr (DUAL) {
                    // per row tile x in bit x: parities of its tiles and blocks so far, and
                    // whether it has had a tile
                    uint32_t qpar = 0, ppar = 0, had = 0;
                    // the first S of a tile's row tile x, of nx blocks, from the K unit at p
                    auto first_qk = [&](int x, int nx, Pos p, bool wait) {
                        if (nx == 0 || !ok) return;
                        ok = (!wait || full(p)) && sleep_wait(&bars[Y::B_Q + x], (qpar >> x) & 1, abort, err);
                        if (!ok) return;
                        tc_fence_after();
                        issue_qk(x, tmem + 128u * x, p, 0);
                        mma_commit_w(&bars[Y::B_S + x]);
                        if (nx == 1) mma_commit_w(&bars[Y::B_QFREE + x]);
                    };
                    Tile t = info(0, false);
                    int n0 = uniform(rows_of(t, 0, tok0, ntok)), n1 = uniform(rows_of(t, 1, tok0, ntok));
                    if (max(n0, n1) > 0) {
                        first_qk(0, n0, pos, true);
                        first_qk(1, n1, pos, n0 == 0);
                        if (ok) freed(pos);
                    }
                    for (int r = 0; ok && t.seq >= 0; ++r) {
                        const int n = max(n0, n1);
                        // units of the tile: K0 (done), V0 K1 V1 K2 ... V(n-1), then K0 of the next one
                        t = info(r + 1, false);
                        const int m0 = uniform(rows_of(t, 0, tok0, ntok)), m1 = uniform(rows_of(t, 1, tok0, ntok));
                        const bool more = max(m0, m1) > 0;
                        if (n == 0 && more) {  // (a tile without keys)
                            first_qk(0, m0, pos, true);
                            first_qk(1, m1, pos, m0 == 0);
                            if (ok) freed(pos);
                        }
                        for (int j = 0; j < n && ok; ++j) {
                            const Pos pv = pos.next(), pk = pv.next();
                            const bool last = j == n - 1;
                            // row tile x: P.V of block j, S of block j + 1 (or of the next tile's first)
                            auto step = [&](auto xc) {
                                constexpr int x = decltype(xc)::value;
                                if (!ok) return;
                                const int nx = x == 0 ? n0 : n1;
                                if (j < nx) {
                                    if (x == 0 || j >= n0) ok = full(pv);
                                    if (j == 0) {
                                        if ((had >> x) & 1)  // the output of the tile before has been read
                                            ok = ok && sleep_wait(&bars[Y::B_OFREE + x], ((qpar >> x) & 1) ^ 1, abort, err);
                                        had |= 1u << x;
                                        qpar ^= 1u << x;
                                    }
                                    ok = ok && sleep_wait(&bars[Y::B_P + x], (ppar >> x) & 1, abort, err);
                                    if (!ok) return;
                                    ppar ^= 1u << x;
                                    tc_fence_after();
                                    issue_pv(tmem + Y::TM_O + (uint32_t)(D * x), tmem + 128u * x, pv, 0, j == 0);
                                    if (j + 1 == nx) mma_commit_w(&bars[Y::B_O + x]);
                                }
                                if (x == 1) freed(pv);  // both row tiles are past V(j)
                                if (!last) {
                                    if (j + 1 < nx) {
                                        if (x == 0 || j + 1 >= n0) ok = full(pk);
                                        if (!ok) return;
                                        tc_fence_after();
                                        issue_qk(x, tmem + 128u * x, pk, 0);
                                        mma_commit_w(&bars[Y::B_S + x]);
                                        if (j + 2 == nx) mma_commit_w(&bars[Y::B_QFREE + x]);
                                    }
                                } else if (more) {
                                    first_qk(x, x == 0 ? m0 : m1, pk, x == 0 || m0 == 0);
                                }
                            };
                            step(std::integral_constant<int, 0>());
                            step(std::integral_constant<int, 1>());
                            if (ok && (!last || more)) freed(pk);
                            pos = pk;
                        }
                        n0 = m0;
                        n1 = m1;
                        warp_arrive(&bars[Y::B_INFOFREE + r % NINFO]);
                    }
                } else {
                    int nt = 0, nb = 0;  // tiles with keys and blocks so far
                    for (int r = 0; ok; ++r) {
                        const Tile t = info(r, false);
                        if (t.seq < 0) break;
                        const int n = uniform(rows_of(t, 0, tok0, ntok));
                        auto qk = [&](int j) -> bool {  // units in order: K0 K1 V0 K2 V1 ... V(n-1)
#pragma unroll
                            for (int h = 0; h < NU; ++h) {
                                if (!full(pos)) return false;
                                tc_fence_after();
                                issue_qk(0, tmem + 128u * ((nb + j) & 1), pos, h);
                                freed(pos);
                                pos = pos.next();
                            }
                            mma_commit_w(&bars[Y::B_S + ((nb + j) & 1)]);
                            if (j == n - 1) mma_commit_w(&bars[Y::B_QFREE]);
                            return true;
                        };
                        if (n > 0) {
                            ok = sleep_wait(&bars[Y::B_Q], nt & 1, abort, err);
                            if (ok) ok = qk(0);
                            for (int j = 0; j < n && ok; ++j) {
                                if (j + 1 < n && !(ok = qk(j + 1))) break;
                                if (j == 0 && nt > 0)  // the output of the tile before has been read
                                    ok = sleep_wait(&bars[Y::B_OFREE], (nt - 1) & 1, abort, err);
                                const int b = nb + j;
                                ok = ok && sleep_wait(&bars[Y::B_P + (b & 1)], (b >> 1) & 1, abort, err);
                                if (!ok) break;
#pragma unroll
                                for (int h = 0; h < NU; ++h) {
                                    ok = ok && full(pos);
                                    if (!ok) break;
                                    tc_fence_after();
                                    issue_pv(tmem + Y::TM_O, tmem + 128u * (b & 1), pos, h, j == 0);
                                    freed(pos);
                                    pos = pos.next();
                                }
                                mma_commit_w(&bars[Y::B_O]);
                            }
                            ++nt;
                            nb += n;
                        }
                        warp_arrive(&bars[Y::B_INFOFREE + r % NINFO]);
                    }
                }
                mma_commit_w(&bars[Y::B_DONE]);
                if (lane == 0) (void)mbar_wait_bounded(&bars[Y::B_DONE], 0, nullptr);
            }
            __syncwarp();
        }
        if (warp == W_LOOK) {
            // ================================================== values on the diagonal
            constexpr int KEYS = BN / NU;
            int u = 0;
            bool ok = true;
            for (int r = 0; ok; ++r) {
                const Tile t = info(r, false);
                if (t.seq < 0) break;
                int tok0[2], ntok[2], nblk[2] = {0, 0}, from = 0x7FFFFFFF;
#pragma unroll
                for (int x = 0; x < QT; ++x) {
                    nblk[x] = rows_of(t, x, tok0[x], ntok[x]);
                    // the first block that the row tile's first row does not see all of
                    if (nblk[x] > 0 && P.causal) from = min(from, max(0, min(t.lk, t.lk - t.lq + tok0[x] + 1)) / BN);
                }
                const int n = max(nblk[0], nblk[1]);
                uint32_t odd = 0;
                for (int v = 0; v < 2 * n * NU && ok; ++v, ++u) {
                    bool isv;
                    int j, half;
                    unit_of(v, n, isv, j, half);
                    const int slot = u % NS;
                    ok = sleep_wait(&bars[Y::B_FULL + slot], (u / NS) & 1, abort, err);
                    if (!ok) break;
                    if (isv && j >= from) {
                        const int rows = min(KEYS, t.lk - j * BN - half * KEYS);
                        // a 16-byte word of 8 values: adding one to the exponents carries into the
                        // sign place when they are all ones
                        constexpr uint32_t ONE = BF16 ? 0x00800080u : 0x04000400u;
                        for (int i = lane; i < rows * 8; i += 32) {
#pragma unroll
                            for (int pn = 0; pn < Y::PANELS; ++pn) {
                                const uint4 w = *reinterpret_cast<const uint4 *>(smem + Y::KV_OFF + slot * Y::UNIT +
                                                                                 pn * KEYS * 128 + i * 16);
                                odd |= ((w.x & 0x7FFF7FFFu) + ONE) | ((w.y & 0x7FFF7FFFu) + ONE) |
                                       ((w.z & 0x7FFF7FFFu) + ONE) | ((w.w & 0x7FFF7FFFu) + ONE);
                            }
                        }
                    }
                    warp_arrive(&bars[Y::B_FREE + slot]);
                }
                if (!ok) break;
                odd = __any_sync(0xffffffffu, (odd & 0x80008000u) != 0);
                if (lane == 0) reinterpret_cast<int *>(smem + Y::INFO_OFF + (r % NINFO) * 32)[7] = (int)odd;
                warp_arrive(&bars[Y::B_LOOK + r % NINFO]);
                warp_arrive(&bars[Y::B_INFOFREE + r % NINFO]);
            }
        }
    } else {
        // ================================================== softmax and output
        regs_inc<REGS_SOFTMAX>();
        const int wg = warp >> 2, qd = warp & 3;
        const int x = DUAL ? wg : 0;
        const int r = 32 * qd + lane;  // row of the tile = tensor-memory lane
        const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16);
        const int ti = r / P.G, hg = r % P.G;
        const float c = P.softmax_scale * LOG2E;
        const uint64_t c2 = f2(c, c);
        constexpr int NCOL = Y::NCOL;
        const int col0 = DUAL ? 0 : 64 * wg;
        const uint32_t tO = tl + Y::TM_O + (DUAL ? (uint32_t)(D * x) : (uint32_t)(128 * wg));
        constexpr int OC = DUAL ? D : 128;  // output channels this thread handles
        bool ok = true;
        int wphase = 0, nb = 0, no = 0, u = 0;  // exchanges, blocks, tiles with keys (of this row tile), ring unit
        int rd = 0;
        // one row of the output: o(i) gives 32 channels
        // (32-byte stores where the base allows them: whole sectors, half the instructions)
        const bool wide = (reinterpret_cast<uintptr_t>(P.out) & 31) == 0;
        auto write_row = [&](size_t row, int i, const float *o) {
            const size_t e0 = row * D + (DUAL ? 0 : 128 * wg) + 32 * i;
            uint32_t w[32];
            const bool f32 = P.out_dtype == PA_F32;
            if (f32) {
#pragma unroll
                for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e]);
            } else if (P.out_dtype == PA_BF16) {
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = pack_f16x2(o[2 * e], o[2 * e + 1]);
            }
            uint8_t *d = static_cast<uint8_t *>(P.out) + e0 * (f32 ? 4 : 2);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (e >= 2 && !f32) break;
                if (wide) {
                    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(d + 32 * e), "r"(w[8 * e]),
                                 "r"(w[8 * e + 1]), "r"(w[8 * e + 2]), "r"(w[8 * e + 3]), "r"(w[8 * e + 4]),
                                 "r"(w[8 * e + 5]), "r"(w[8 * e + 6]), "r"(w[8 * e + 7])
                                 : "memory");
                } else {
                    *reinterpret_cast<uint4 *>(d + 32 * e) = make_uint4(w[8 * e], w[8 * e + 1], w[8 * e + 2], w[8 * e + 3]);
                    *reinterpret_cast<uint4 *>(d + 32 * e + 16) =
                        make_uint4(w[8 * e + 4], w[8 * e + 5], w[8 * e + 6], w[8 * e + 7]);
                }
            }
        };
        for (;; ++rd) {
            // what the blocks need: their number; the ring units of the tile; the keys this
            // row sees; the first block that some row does not see all of; the block
            // whose V rows past the sequence this warpgroup zeroes
            int nblk, n, vis, jmask, jzero;
            {
                const Tile t = info(rd, false);
                if (t.seq < 0) break;
                int t0, ntok, a, b;
                nblk = rows_of(t, x, t0, ntok);
                const int other = DUAL ? rows_of(t, 1 - x, a, b) : nblk, nblk0 = x == 0 ? nblk : other;
                n = max(nblk, other);
                const int off = t.lk - t.lq;
                const bool live = ti < ntok && ti < P.tpt;
                vis = !live ? 0 : P.causal ? max(0, min(t.lk, off + t0 + ti + 1)) : t.lk;
                jmask = (P.causal ? max(0, min(t.lk, off + t0 + 1)) : t.lk) / BN;
                jzero = t.lk % BN != 0 && (!DUAL || x == 0 || t.lk / BN >= nblk0) ? t.lk / BN : -1;
            }
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < nblk; ++j, ++nb) {
                const uint32_t tS = tl + 128u * (DUAL ? x : (nb & 1));
                ok = sleep_wait(&bars[Y::B_S + (DUAL ? x : (nb & 1))], (DUAL ? nb : (nb >> 1)) & 1, abort, err);
                if (!ok) break;
                tc_fence_after();
                float s[NCOL];
#pragma unroll
                for (int i = 0; i < NCOL / 32; ++i) tmem_ld32_nowait(tS + (uint32_t)(col0 + 32 * i), s + 32 * i);
#pragma unroll
                for (int i = 0; i < NCOL / 32; ++i) tmem_wait32(s + 32 * i);
                if (j >= jmask) {
                    const int lim = vis - j * BN - col0;  // columns of this row that count
#pragma unroll
                    for (int q = 0; q < NCOL; q += 32)
                        if (!__all_sync(0xffffffffu, lim >= q + 32)) {
#pragma unroll
                            for (int i = q; i < q + 32; ++i) s[i] = i < lim ? s[i] : -INFINITY;
                        }
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int i = 4; i < NCOL; i += 8) {
                    mx[0] = fmaxf(fmaxf(mx[0], s[i]), s[i + 1]);
                    mx[1] = fmaxf(fmaxf(mx[1], s[i + 2]), s[i + 3]);
                    if (i + 4 < NCOL) {
                        mx[2] = fmaxf(fmaxf(mx[2], s[i + 4]), s[i + 5]);
                        mx[3] = fmaxf(fmaxf(mx[3], s[i + 6]), s[i + 7]);
                    }
                }
                float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if constexpr (!DUAL) {
                    // both halves of the row agree on its maximum; two buffers, since a
                    // warp may start the next exchange before its partner read this one
                    // (the one after that waits for the partner's next arrival)
                    float *rb = red + (wphase & 1) * 256;
                    rb[wg * 128 + r] = mb;
                    warp_arrive(&bars[Y::B_WG]);
                    ok = sleep_wait(&bars[Y::B_WG], wphase & 1, abort, err);
                    ++wphase;
                    if (!ok) break;
                    mb = fmaxf(mb, rb[(wg ^ 1) * 128 + r]);
                }
                if (__any_sync(0xffffffffu, (mb - m) * c > SLACK || (m == -INFINITY && mb > m))) {
                    const float mn = fmaxf(m, mb);
                    const float f = mn == -INFINITY ? 1.f : ex2((m - mn) * c);
                    m = mn;
                    l *= f;
                    if (j > 0) {
                        if constexpr (!DUAL) {
                            // the previous block's P.V must be complete (with two row
                            // tiles it is: S of this block was issued after it)
                            ok = sleep_wait(&bars[Y::B_O], (nb - 1) & 1, abort, err);
                            if (!ok) break;
                            tc_fence_after();
                        }
#pragma unroll 1
                        for (int i = 0; i < OC / 16; ++i) {
                            float o[16];
                            tmem_ld16_nowait(tO + 16u * i, reinterpret_cast<uint32_t *>(o));
                            tmem_wait16(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= f;
                            tmem_st16_u(tO + 16u * i, reinterpret_cast<const uint32_t *>(o));
                        }
                        tmem_st_wait();
                    }
                }
                const float mc = m == -INFINITY ? 0.f : m * c;
                const uint64_t nm2 = f2(-mc, -mc);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int q = 0; q < NCOL / 64; ++q) {
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float a, b;
                        f2_split(fma2(f2(s[64 * q + 2 * i], s[64 * q + 2 * i + 1]), c2, nm2), a, b);
                        a = ex2(a);
                        b = ex2(b);
                        sum[i & 3] = add2(sum[i & 3], f2(a, b));
                        pk[i] = pack2<BF16>(a, b);
                    }
                    tmem_st32_u(tS + (uint32_t)(col0 / 2 + 32 * q), pk);
                }
                {
                    const uint64_t t2 = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                    float a, b;
                    f2_split(t2, a, b);
                    l += a + b;
                }
                // V rows past the sequence (the next one's, whatever they hold) are
                // zeroed before the product: 0 * NaN would be NaN
                if (j == jzero) {
                    const int tail = entry(rd).lk - j * BN, tt = DUAL ? (j << 1 | 1) : (j == n - 1 ? 2 * n - 1 : 2 * j + 2);
                    const int ti2 = DUAL ? r : (wg << 7 | r);
                    constexpr int NT = DUAL ? 128 : 256, KEYS = BN / NU;
                    for (int hf = 0; hf < NU && ok; ++hf) {
                        const int uu = u + tt * NU + hf;
                        ok = sleep_wait(&bars[Y::B_FULL + uu % NS], (uu / NS) & 1, abort, err);
                        if (!ok) break;
                        const int from = max(0, tail - hf * KEYS);
                        uint8_t *vt = smem + Y::KV_OFF + (uu % NS) * Y::UNIT;
                        const int words = max(0, KEYS - from) * 8;
                        for (int i = ti2; i < words * Y::PANELS; i += NT) {
                            const int pn = i / words, w = i - pn * words;
                            *reinterpret_cast<uint4 *>(vt + pn * KEYS * 128 + from * 128 + w * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    if (!ok) break;
                    fence_proxy_async_smem();
                }
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(&bars[Y::B_P + (DUAL ? x : (nb & 1))]);
            }
            if (!ok) break;
            u += 2 * n * NU;
            // ---- output rows
            ok = sleep_wait(&bars[Y::B_LOOK + rd % NINFO], (rd / NINFO) & 1, abort, err);
            if (!ok) break;
            if (nblk > 0) {
                ok = DUAL ? sleep_wait(&bars[Y::B_O + x], no & 1, abort, err)
                          : sleep_wait(&bars[Y::B_O], (nb - 1) & 1, abort, err);
                ++no;
                if constexpr (!DUAL) {
                    if (ok) {
                        float *rb = red + (wphase & 1) * 256;
                        rb[wg * 128 + r] = l;
                        warp_arrive(&bars[Y::B_WG]);
                        ok = sleep_wait(&bars[Y::B_WG], wphase & 1, abort, err);
                        ++wphase;
                        if (ok) l = wg == 0 ? l + rb[128 + r] : rb[r] + l;
                    }
                }
                if (!ok) break;
                tc_fence_after();
            }
            const Tile t = entry(rd);
            int t0, ntok;
            (void)rows_of(t, x, t0, ntok);
            const bool live = ti < ntok && ti < P.tpt;  // (rows past 128 / G * G, or past the sequence, are not written)
            const size_t row = (size_t)(t.q0 + t0 + ti) * P.Hq + t.g * P.G + hg;
            const bool nan_row = t.lk < 0;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (live && P.lse != nullptr && (DUAL || wg == 0))
                P.lse[row] = nan_row ? NaN : l == 0.f ? -INFINITY : m * P.softmax_scale + logf(l);
            const bool again =
                reinterpret_cast<const volatile int *>(smem + Y::INFO_OFF + (rd % NINFO) * 32)[7] != 0 && nblk > 0;
            if (again) {
                // values that are not finite beside masked keys: row by row over the
                // visible keys (head dim 256: by the first warpgroup), lanes over channels
                tc_fence_before();
                warp_arrive(&bars[Y::B_OFREE + x]);
                constexpr int CL = D / 32;
                auto val = [](uint16_t b) {
                    return BF16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
                };
#pragma unroll 1
                for (int rr = 0; rr < 32; ++rr) {
                    const int vr = __shfl_sync(0xffffffffu, vis, rr);
                    const float mr = __shfl_sync(0xffffffffu, m, rr), ir = __shfl_sync(0xffffffffu, inv, rr);
                    const bool lr = __shfl_sync(0xffffffffu, (int)live, rr) != 0;
                    const size_t rowr = __shfl_sync(0xffffffffu, (unsigned long long)row, rr);
                    if (!lr || (!DUAL && wg != 0)) continue;
                    float q[CL], o[CL];
                    const size_t qrow = rowr / P.Hq, qh = rowr % P.Hq;
#pragma unroll
                    for (int e = 0; e < CL; ++e) {
                        q[e] = val(P.q[qrow * P.qs + qh * D + lane * CL + e]);
                        o[e] = 0.f;
                    }
                    const float mcr = mr == -INFINITY ? 0.f : mr * c;
#pragma unroll 1
                    for (int key = 0; key < vr; ++key) {
                        const uint16_t *kr = P.k + (size_t)(t.k0 + key) * P.ks + (size_t)t.g * D + lane * CL;
                        const uint16_t *vv = P.v + (size_t)(t.k0 + key) * P.vs + (size_t)t.g * D + lane * CL;
                        float z = 0.f;
#pragma unroll
                        for (int e = 0; e < CL; ++e) z = fmaf(q[e], val(kr[e]), z);
#pragma unroll
                        for (int off = 16; off >= 1; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
                        const float pz = ex2(fmaf(z, c, -mcr));
#pragma unroll
                        for (int e = 0; e < CL; ++e) o[e] = fmaf(pz, val(vv[e]), o[e]);
                    }
#pragma unroll
                    for (int e = 0; e < CL; ++e) {
                        const float y = ir == 0.f ? 0.f : o[e] * ir;
                        const size_t at = rowr * D + lane * CL + e;
                        if (P.out_dtype == PA_F32) reinterpret_cast<float *>(P.out)[at] = y;
                        else if (P.out_dtype == PA_BF16) reinterpret_cast<__nv_bfloat16 *>(P.out)[at] = __float2bfloat16_rn(y);
                        else reinterpret_cast<__half *>(P.out)[at] = __float2half_rn(y);
                    }
                }
            } else {
                // (a row that saw nothing: inv = 0, and its sums are 0)
                const uint64_t inv2 = f2(inv, inv);
                const float fill = nan_row ? NaN : 0.f;
#pragma unroll 1
                for (int i = 0; i < OC / 32; ++i) {
                    float o[32];
                    if (nblk > 0) {
                        tmem_ld32_nowait(tO + 32u * i, o);
                        tmem_wait32(o);
                        if (i == OC / 32 - 1) {  // O may be overwritten by the next tile
                            tc_fence_before();
                            warp_arrive(&bars[Y::B_OFREE + x]);
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2) f2_split(mul2(f2(o[e], o[e + 1]), inv2), o[e], o[e + 1]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = fill;
                    }
                    if (live) write_row(row, i, o);
                    __syncwarp();
                }
            }
            warp_arrive(&bars[Y::B_INFOFREE + rd % NINFO]);
        }
        warp_arrive(&bars[Y::B_EXIT]);
    }

    // ---- teardown
    if (err) atomicOr(reinterpret_cast<unsigned *>(misc + 2), err);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W_MMA)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Y::TM_COLS) : "memory");
    if (tid == 0 && misc[2] != 0 && P.dev_error) atomicOr(P.dev_error, (uint32_t)misc[2]);
}

template <int D, bool BF16>
cudaError_t launch_prompt(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const PromptParams &P,
                          long long tiles, cudaStream_t s) {
    // the attribute is per device; setting it again is harmless, so a plain flag per device suffices
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev >= 64 || !(done.load(std::memory_order_relaxed) & bit)) {
        // the register split draws on what the block was launched with
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, pa_prompt_kernel<D, BF16>);
        if (e != cudaSuccess) return e;
        if (at.numRegs < REGS_LAUNCH) return cudaErrorLaunchOutOfResources;
        e = cudaFuncSetAttribute(pa_prompt_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::SMEM);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const unsigned ctas = (unsigned)std::min<long long>(sms, tiles);
    // a grid that leaves SMs free may set up on them while the kernel before drains
    // (two short prompts 7.8 us a call, 9.9 without); one that fills them gains nothing
    if ((int)ctas < sms)
        return launch_pdl(pa_prompt_kernel<D, BF16>, dim3(ctas), dim3(THREADS), Lay<D>::SMEM, s, tq, tk, tv, P);
    pa_prompt_kernel<D, BF16><<<ctas, THREADS, Lay<D>::SMEM, s>>>(tq, tk, tv, P);
    return cudaPeekAtLastError();
}

}  // namespace prompt
}  // namespace pa

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

bool encode4(CUtensorMap *tm, int dtype, const void *base, const cuuint64_t *dims, const cuuint64_t *strides,
             const cuuint32_t *box) {
    auto enc = encode_fn();
    if (enc == nullptr) return false;
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(tm, dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
               const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// rows of [heads][D], `stride` elements apart: boxes of 64 channels of `rows` keys of one head
bool encode_kv(CUtensorMap *tm, const pa_prompt_problem *p, const void *base, long long stride, int rows) {
    const cuuint64_t dims[4] = {(cuuint64_t)p->head_dim, (cuuint64_t)p->total_k, (cuuint64_t)p->num_kv_heads, 1};
    const cuuint64_t strides[3] = {(cuuint64_t)stride * 2, (cuuint64_t)p->head_dim * 2,
                                   (cuuint64_t)p->head_dim * 2 * p->num_kv_heads};
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
    return encode4(tm, p->dtype, base, dims, strides, box);
}

}  // namespace

extern "C" PA_API pa_status pa_prompt_attention(const pa_prompt_problem *p, const void *q, const void *k, const void *v,
                                                const int32_t *cu_q, const int32_t *cu_k, void *out, float *lse,
                                                uint32_t *dev_error, pa_stream_t stream) {
    if (p == nullptr) return PA_ERR_INVALID_ARG;
    if (p->num_seqs < 0 || p->total_q < 0 || p->total_k < 0 || p->num_q_heads < 1 || p->num_kv_heads < 1 ||
        p->num_q_heads % p->num_kv_heads != 0 || p->head_dim < 1 || p->q_stride < 0 || p->k_stride < 0 ||
        p->v_stride < 0)
        return PA_ERR_INVALID_ARG;
    if ((p->dtype != PA_F16 && p->dtype != PA_BF16) ||
        (p->out_dtype != PA_F32 && p->out_dtype != PA_F16 && p->out_dtype != PA_BF16) ||
        (p->causal != 0 && p->causal != 1) || !std::isfinite(p->softmax_scale) || p->softmax_scale <= 0.f)
        return PA_ERR_INVALID_ARG;
    const int D = p->head_dim, G = p->num_q_heads / p->num_kv_heads;
    const long long qrow = (long long)p->num_q_heads * D, krow = (long long)p->num_kv_heads * D;
    const long long qs = p->q_stride ? p->q_stride : qrow, ks = p->k_stride ? p->k_stride : krow,
                    vs = p->v_stride ? p->v_stride : krow;
    if (qs < qrow || ks < krow || vs < krow) return PA_ERR_INVALID_ARG;
    if ((D != 64 && D != 128 && D != 256) || G > 128 || p->num_seqs > 65535 || qs % 8 || ks % 8 || vs % 8)
        return PA_ERR_UNSUPPORTED;
    const int tpt = 128 / G, tq_tokens = D == 256 ? tpt : 2 * tpt;
    // tiles at most: every sequence rounds up once
    const long long tiles = ((long long)p->total_q / tq_tokens + std::min(p->num_seqs, p->total_q)) * p->num_kv_heads;
    if (tiles > 0x7FFFFFFFll) return PA_ERR_UNSUPPORTED;
    if (p->num_seqs == 0 || p->total_q == 0) return PA_OK;
    if (q == nullptr || cu_q == nullptr || cu_k == nullptr || out == nullptr ||
        (p->total_k > 0 && (k == nullptr || v == nullptr)))
        return PA_ERR_INVALID_ARG;
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(out, 16) || misaligned(lse, 4) ||
        misaligned(cu_q, 4) || misaligned(cu_k, 4) || misaligned(dev_error, 4))
        return PA_ERR_INVALID_ARG;

    CUtensorMap tq, tk, tv;
    {
        // channels, heads of the group, tokens, kv heads
        const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)G, (cuuint64_t)p->total_q, (cuuint64_t)p->num_kv_heads};
        const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)qs * 2, (cuuint64_t)G * D * 2};
        const cuuint32_t box[4] = {64, (cuuint32_t)G, (cuuint32_t)tpt, 1};
        if (!encode4(&tq, p->dtype, q, dims, strides, box)) return PA_ERR_CUDA;
    }
    if (p->total_k > 0) {
        if (!encode_kv(&tk, p, k, ks, 128) || !encode_kv(&tv, p, v, vs, D == 256 ? 64 : 128)) return PA_ERR_CUDA;
    } else {
        tk = tq;  // no keys: never read
        tv = tq;
    }
    pa::PromptParams P;
    P.cu_q = cu_q;
    P.cu_k = cu_k;
    P.out = out;
    P.lse = lse;
    P.dev_error = dev_error;
    P.B = p->num_seqs;
    P.total_q = p->total_q;
    P.total_k = p->total_k;
    P.Hq = p->num_q_heads;
    P.Hkv = p->num_kv_heads;
    P.G = G;
    P.tpt = tpt;
    P.max_tiles = (int)(tiles / p->num_kv_heads);
    P.tq_mul = tq_tokens > 1 ? (unsigned)((1ull << 32) / (unsigned)tq_tokens) + 1u : 0u;
    P.out_dtype = p->out_dtype;
    P.causal = p->causal;
    P.q = static_cast<const uint16_t *>(q);
    P.k = static_cast<const uint16_t *>(k);
    P.v = static_cast<const uint16_t *>(v);
    P.qs = qs;
    P.ks = ks;
    P.vs = vs;
    P.softmax_scale = p->softmax_scale;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    const bool bf = p->dtype == PA_BF16;
    switch (D) {
        case 64: e = bf ? pa::prompt::launch_prompt<64, true>(tq, tk, tv, P, tiles, s)
                        : pa::prompt::launch_prompt<64, false>(tq, tk, tv, P, tiles, s); break;
        case 128: e = bf ? pa::prompt::launch_prompt<128, true>(tq, tk, tv, P, tiles, s)
                         : pa::prompt::launch_prompt<128, false>(tq, tk, tv, P, tiles, s); break;
        default: e = bf ? pa::prompt::launch_prompt<256, true>(tq, tk, tv, P, tiles, s)
                        : pa::prompt::launch_prompt<256, false>(tq, tk, tv, P, tiles, s); break;
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
