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
// Tiles are independent CTAs, handed out longest first: tile i of the grid is
// found by counting, for a bisected number of key blocks c, how many tiles
// visit at least c blocks (a closed form per sequence), so no plan kernel and
// no workspace are needed and the block scheduler balances the load.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "pa_attn.cuh"
#include "pa_tc.cuh"

namespace pa {

struct PromptParams {
    const int32_t *cu_q;
    const int32_t *cu_k;
    void *out;
    float *lse;
    uint32_t *dev_error;
    int B, total_q, total_k, Hq, Hkv, G;
    int tpt;     // query tokens per 128-row tile: 128 / G
    int out_dtype, causal;
    float softmax_scale;
};

namespace prompt {

using namespace tc;

constexpr int BN = 128;                 // keys per block
constexpr float SLACK = 8.0f;           // exp2-domain headroom of the lazy maximum
constexpr int W_LOAD = 8, W_MMA = 9;    // warps 0-3, 4-7: softmax
constexpr int THREADS = 384;            // warps 10, 11 idle: the warpgroup gives its registers to the softmax
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
        B_FULL = B_Q + 2,        // [NS]
        B_FREE = B_FULL + NS,    // [NS]
        B_S = B_FREE + NS,       // [2] S complete (per tile, or per buffer)
        B_P = B_S + 2,           // [2] P written, O rescaled
        B_O = B_P + 2,           // [2] dual: the tile's last P.V complete; else [0] every P.V
        B_WG = B_O + 2,          // the eight softmax warps (D = 256)
        B_DONE = B_WG + 1,
        NBARS = B_DONE + 1
    };
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;  // [0] tmem, [1] abort, [2] errors, [8..] tile search
    static constexpr int SMEM = MISC_OFF + 256;
    static constexpr int TM_O = 256, TM_COLS = 512;
    static_assert(SMEM <= 227 * 1024, "prompt kernel exceeds the shared memory of one CTA");
};

struct Seq {
    int q0, lq, k0, lk;  // lk < 0: the key range breaks the contract; lq = 0 when the query range does
    bool bad;
};

__device__ __forceinline__ Seq load_seq(const PromptParams &P, int s) {
    Seq r;
    const int a = P.cu_q[s], b = P.cu_q[s + 1], c = P.cu_k[s], d = P.cu_k[s + 1];
    const bool okq = a >= 0 && a <= b && b <= P.total_q, okk = c >= 0 && c <= d && d <= P.total_k;
    r.q0 = a;
    r.lq = okq ? b - a : 0;
    r.k0 = c;
    r.lk = okk ? d - c : -1;
    r.bad = !okq || !okk;
    return r;
}

// tiles of `tq` query tokens that visit at least c blocks of keys: the last
// `count` of the sequence's nt tiles (blocks grow with the tile)
__device__ __forceinline__ int tiles_with(int lq, int lk, int c, int tq, int causal) {
    const int nt = (lq + tq - 1) / tq;
    if (c <= 0) return nt;
    const int need = (c - 1) * BN;  // visible keys of the tile's last row must exceed this
    if (lk <= need) return 0;
    if (!causal) return nt;
    const int x = need - (lk - lq);
    const int first = x < 0 ? 0 : min(x / tq, nt - 1);
    return nt - first;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS, 1)
    pa_prompt_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv, PromptParams P) {
    using Y = Lay<D>;
    constexpr bool DUAL = Y::DUAL;
    constexpr int NS = Y::NS, NU = Y::NU;
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
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float NaN = __int_as_float(0x7fc00000);

    // ---- which tile: counts of tiles by blocks visited, bisected
    const int TQ = P.tpt * Y::QT;
    const int g = blockIdx.x % P.Hkv;
    const int want = blockIdx.x / P.Hkv;
    int seq = 0, tile = 0;
    if (tid < 48) misc[8 + tid] = 0;
    if (tid == 0) {
        misc[1] = 0;
        misc[2] = 0;
    }
    __syncthreads();
    bool bad = false;
    {
        // sums over the sequences, one shared counter per question asked
        int asked = 0;
        auto total_with = [&](int c) -> int {
            int n = 0;
            for (int s = tid; s < P.B; s += THREADS) {
                const Seq q = load_seq(P, s);
                bad |= q.bad;
                n += tiles_with(q.lq, q.lk, c, TQ, P.causal);
            }
            n = __reduce_add_sync(0xffffffffu, n);
            int *slot = misc + 8 + asked++;
            if (lane == 0 && n) atomicAdd(slot, n);
            __syncthreads();
            return *slot;
        };
        if (want >= total_with(0)) {
            if (blockIdx.x == gridDim.x - 1 && bad && P.dev_error) atomicOr(P.dev_error, PA_DEV_ERR_CONTEXT_LEN);
            return;  // the grid is sized from totals: some CTAs have no tile
        }
        int lo = 0, hi = (P.total_k + BN - 1) / BN + 1, above = 0;  // count(lo) > want >= count(hi) = above
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            const int n = total_with(mid);
            if (n > want) lo = mid;
            else {
                hi = mid;
                above = n;
            }
        }
        // the (want - above)-th tile, by sequence, of those with exactly lo blocks
        const int rank = want - above;
        if (warp == 0) {
            int before = 0;
            for (int base = 0; base < P.B; base += 32) {
                const int s = base + lane;
                int n = 0, first = 0;
                if (s < P.B) {
                    const Seq q = load_seq(P, s);
                    const int ge = tiles_with(q.lq, q.lk, lo, TQ, P.causal);
                    const int gt = tiles_with(q.lq, q.lk, lo + 1, TQ, P.causal);
                    n = ge - gt;
                    first = (q.lq + TQ - 1) / TQ - ge;
                }
                int x = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                const int ex = before + x - n;
                const bool mine = rank >= ex && rank < ex + n;
                if (mine) {
                    misc[3] = s;
                    misc[4] = first + rank - ex;
                }
                if (__any_sync(0xffffffffu, mine)) break;
                before += __shfl_sync(0xffffffffu, x, 31);
            }
        }
        __syncthreads();
        seq = misc[3];
        tile = misc[4];
        if (bad && want == 0 && P.dev_error) atomicOr(P.dev_error, PA_DEV_ERR_CONTEXT_LEN);
    }
    const Seq sq = load_seq(P, seq);
    const int off = sq.lk - sq.lq;
    // per row tile: first token, tokens, blocks of keys
    int tok0[2], ntok[2], nblk[2] = {0, 0};
#pragma unroll
    for (int x = 0; x < Y::QT; ++x) {
        tok0[x] = (tile * Y::QT + x) * P.tpt;
        ntok[x] = min(P.tpt, sq.lq - tok0[x]);
        if (ntok[x] > 0 && sq.lk > 0) {
            const int vis = P.causal ? min(sq.lk, off + tok0[x] + ntok[x]) : sq.lk;
            nblk[x] = vis > 0 ? (vis + BN - 1) / BN : 0;
        }
    }
    const int n = max(nblk[0], nblk[1]);

    if (tid == 0) {
        for (int i = 0; i < Y::NBARS; ++i) {
            uint32_t c = 1;
            if (i >= Y::B_P && i < Y::B_P + 2) c = DUAL ? 4 : 8;
            if (i == Y::B_WG) c = 8;
            mbar_init(&bars[i], c);
        }
        mbar_fence_init();
    }
    if (warp == W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + Y::MISC_OFF),
                     "r"(Y::TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)misc[0];
    uint32_t err = 0;

    if (warp >= W_LOAD) {
    regs_dec<REGS_OTHER>();  // the whole third warpgroup
    if (warp == W_LOAD) {
        // ================================================== tensor copies
        if (lane == 0 && n > 0) {
            const uint32_t qbytes = (uint32_t)(P.tpt * P.G) * 128u * Y::PANELS;
#pragma unroll
            for (int x = 0; x < Y::QT; ++x) {
                if (nblk[x] == 0) continue;
                mbar_arrive_expect_tx(&bars[Y::B_Q + x], qbytes);
#pragma unroll
                for (int c = 0; c < Y::PANELS; ++c)
                    tma_load_4d(smem + Y::Q_OFF + x * Y::Q_BYTES + c * 128 * 128, &tq, &bars[Y::B_Q + x], 64 * c, 0,
                                sq.q0 + tok0[x], g);
            }
            const int units = 2 * n * NU;
            int u = 0;
            for (; u < units; ++u) {
                const int slot = u % NS;
                if (u >= NS && !sleep_wait<false>(&bars[Y::B_FREE + slot], ((u / NS) - 1) & 1, abort, err)) break;
                const int t = u / NU, half = u % NU;  // tile in the order the products need them
                bool isv;
                int j;
                if (DUAL) {                            // K0 V0 K1 V1 ...
                    isv = t & 1;
                    j = t >> 1;
                } else {                               // K0 K1 V0 K2 V1 ... V(n-1)
                    isv = t > 0 && ((t & 1) == 0 || t == 2 * n - 1);
                    j = t == 0 ? 0 : t == 2 * n - 1 ? n - 1 : isv ? t / 2 - 1 : (t + 1) / 2;
                }
                uint8_t *dst = smem + Y::KV_OFF + slot * Y::UNIT;
                mbar_arrive_expect_tx(&bars[Y::B_FULL + slot], Y::UNIT);
                if (NU == 1) {
#pragma unroll
                    for (int c = 0; c < Y::PANELS; ++c)
                        tma_load_4d(dst + c * BN * 128, isv ? &tv : &tk, &bars[Y::B_FULL + slot], 64 * c,
                                    sq.k0 + j * BN, g, 0);
                } else if (!isv) {                     // channels 128 * half ..: two panels of 128 keys
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tma_load_4d(dst + c * BN * 128, &tk, &bars[Y::B_FULL + slot], 128 * half + 64 * c,
                                    sq.k0 + j * BN, g, 0);
                } else {                               // keys 64 * half ..: four panels of 64 keys
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tma_load_4d(dst + c * 64 * 128, &tv, &bars[Y::B_FULL + slot], 64 * c,
                                    sq.k0 + j * BN + 64 * half, g, 0);
                }
            }
            if (*abort) {  // let every copy still in flight land before the CTA exits
#pragma unroll
                for (int x = 0; x < Y::QT; ++x)
                    if (nblk[x] > 0) (void)mbar_wait_bounded(&bars[Y::B_Q + x], 0, nullptr);
                for (int i = max(0, u - NS); i < u; ++i)
                    (void)mbar_wait_bounded(&bars[Y::B_FULL + i % NS], (i / NS) & 1, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == W_MMA) {
        // ================================================== MMA issue (lane 0 alone)
        constexpr uint32_t FMT = BF16 ? (1u << 7) | (1u << 10) : 0u;
        constexpr uint32_t ID_S = idesc(128, BN, 0) | FMT;
        constexpr uint32_t ID_O = idesc(128, D, 0) | FMT | (1u << 16);  // B = V read MN-major
        auto full = [&](int u) { return sleep_wait<false>(&bars[Y::B_FULL + u % NS], (u / NS) & 1, abort, err); };
        auto kv = [&](int u) { return sb + Y::KV_OFF + (uint32_t)(u % NS) * Y::UNIT; };
        // S = Q K^T over one unit of K (all channels, or 128 of them)
        auto issue_qk = [&](int x, uint32_t dS, int u, int half) {
            const uint64_t a = sdesc(sb + Y::Q_OFF + x * Y::Q_BYTES + half * 2 * 128 * 128, 16, 1024, 2);
            const uint64_t b = sdesc(kv(u), 16, 1024, 2);
            constexpr int STEPS = D / 16 / NU;
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
                const uint32_t o = (uint32_t)((k >> 2) * (128 * 128) + 32 * (k & 3)) >> 4;
                mma_f16(dS, a + o, b + o, ID_S, (half > 0 || k > 0) ? 1u : 0u);
            }
        };
        // O += P V over one unit of V (128 or 64 keys)
        auto issue_pv = [&](uint32_t dO, uint32_t aP, int u, int half, bool first) {
            constexpr int KEYS = BN / NU;
            const uint64_t b = sdesc(kv(u), KEYS * 128, 1024, 2);
#pragma unroll
            for (int k = 0; k < KEYS / 16; ++k)
                mma_f16_ts(dO, aP + (uint32_t)(half * KEYS / 2 + 8 * k), b + (uint32_t)((k * 16 * 128) >> 4), ID_O,
                           (!first || half > 0 || k > 0) ? 1u : 0u);
        };
        if (lane == 0 && n > 0) {
            if constexpr (DUAL) {
                bool ok = full(0);
                for (int x = 0; x < 2 && ok; ++x) {
                    if (nblk[x] == 0) continue;
                    ok = sleep_wait<false>(&bars[Y::B_Q + x], 0, abort, err);
                    if (!ok) break;
                    tc_fence_after();
                    issue_qk(x, tmem + 128u * x, 0, 0);
                    mma_commit(&bars[Y::B_S + x]);
                }
                mma_commit(&bars[Y::B_FREE + 0]);
                for (int j = 0; j < n && ok; ++j) {
                    const int uv = 2 * j + 1, uk = 2 * j + 2;
                    ok = full(uv);
                    for (int x = 0; x < 2 && ok; ++x) {
                        if (j >= nblk[x]) continue;
                        ok = sleep_wait<false>(&bars[Y::B_P + x], j & 1, abort, err);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(tmem + Y::TM_O + (uint32_t)(D * x), tmem + 128u * x, uv, 0, j == 0);
                        if (x == 1 || j >= nblk[1]) mma_commit(&bars[Y::B_FREE + uv % NS]);
                        if (j + 1 < nblk[x]) {
                            ok = full(uk);
                            if (!ok) break;
                            tc_fence_after();
                            issue_qk(x, tmem + 128u * x, uk, 0);
                            mma_commit(&bars[Y::B_S + x]);
                        } else {
                            mma_commit(&bars[Y::B_O + x]);
                        }
                    }
                    if (j + 1 < n) mma_commit(&bars[Y::B_FREE + uk % NS]);
                }
            } else {
                auto qk = [&](int j) -> bool {  // the tile's unit index: K0 = 0, K(j) = 2j - 1
                    const int u0 = (j == 0 ? 0 : 2 * j - 1) * NU;
                    for (int h = 0; h < NU; ++h) {
                        if (!full(u0 + h)) return false;
                        tc_fence_after();
                        issue_qk(0, tmem + 128u * (j & 1), u0 + h, h);
                        mma_commit(&bars[Y::B_FREE + (u0 + h) % NS]);
                    }
                    mma_commit(&bars[Y::B_S + (j & 1)]);
                    return true;
                };
                bool ok = sleep_wait<false>(&bars[Y::B_Q], 0, abort, err);
                if (ok) ok = qk(0);
                for (int j = 0; j < n && ok; ++j) {
                    if (j + 1 < n && !(ok = qk(j + 1))) break;
                    ok = sleep_wait<false>(&bars[Y::B_P + (j & 1)], (j >> 1) & 1, abort, err);
                    if (!ok) break;
                    const int u0 = (j == n - 1 ? 2 * n - 1 : 2 * j + 2) * NU;
                    for (int h = 0; h < NU && ok; ++h) {
                        ok = full(u0 + h);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(tmem + Y::TM_O, tmem + 128u * (j & 1), u0 + h, h, j == 0);
                        mma_commit(&bars[Y::B_FREE + (u0 + h) % NS]);
                    }
                    mma_commit(&bars[Y::B_O]);
                }
            }
            mma_commit(&bars[Y::B_DONE]);
            (void)mbar_wait_bounded(&bars[Y::B_DONE], 0, nullptr);
        }
        __syncwarp();
    }
    } else {
        // ================================================== softmax and output
        regs_inc<REGS_SOFTMAX>();
        const int wg = warp >> 2, qd = warp & 3;
        const int x = DUAL ? wg : 0;
        const int r = 32 * qd + lane;  // row of the tile = tensor-memory lane
        const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16);
        const int nb = x == 0 ? nblk[0] : nblk[1];
        const int t0 = x == 0 ? tok0[0] : tok0[1], nt = x == 0 ? ntok[0] : ntok[1];
        const int ti = r / P.G, h = g * P.G + r % P.G;
        const bool live = ti < nt;     // (rows past 128 / G * G, or past the sequence, are not written)
        const float c = P.softmax_scale * LOG2E;
        const uint64_t c2 = f2(c, c);
        constexpr int NCOL = Y::NCOL;
        const int col0 = DUAL ? 0 : 64 * wg;
        // keys visible to this row, and to every row of the tile
        const int vis = !live ? 0 : P.causal ? max(0, min(sq.lk, off + t0 + ti + 1)) : sq.lk;
        const int vis_all = P.causal ? max(0, min(sq.lk, off + t0 + 1)) : sq.lk;
        const uint32_t tO = tl + Y::TM_O + (DUAL ? (uint32_t)(D * x) : (uint32_t)(128 * wg));
        constexpr int OC = DUAL ? D : 128;  // output channels this thread handles
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        int wphase = 0;
        for (int j = 0; j < nb; ++j) {
            const uint32_t tS = tl + 128u * (DUAL ? x : (j & 1));
            ok = sleep_wait(&bars[Y::B_S + (DUAL ? x : (j & 1))], (DUAL ? j : (j >> 1)) & 1, abort, err);
            if (!ok) break;
            tc_fence_after();
            float s[NCOL];
#pragma unroll
            for (int i = 0; i < NCOL / 32; ++i) tmem_ld32_nowait(tS + (uint32_t)(col0 + 32 * i), s + 32 * i);
#pragma unroll
            for (int i = 0; i < NCOL / 32; ++i) tmem_wait32(s + 32 * i);
            if ((j + 1) * BN > vis_all) {
                const int lim = vis - j * BN - col0;  // columns of this row that count
#pragma unroll
                for (int i = 0; i < NCOL; ++i) s[i] = i < lim ? s[i] : -INFINITY;
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
                        ok = sleep_wait(&bars[Y::B_O], (j - 1) & 1, abort, err);
                        if (!ok) break;
                        tc_fence_after();
                    }
#pragma unroll
                    for (int i = 0; i < OC / 32; ++i) {
                        float o[32];
                        tmem_ld32_nowait(tO + 32u * i, o);
                        tmem_wait32(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f;
                        tmem_st32_u(tO + 32u * i, reinterpret_cast<const uint32_t *>(o));
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
            const int tail = sq.lk - j * BN;
            if (tail < BN && (!DUAL || x == 0 || j >= nblk[0])) {
                const int tt = DUAL ? (j << 1 | 1) : (j == n - 1 ? 2 * n - 1 : 2 * j + 2);
                const int ti2 = DUAL ? r : (wg << 7 | r);
                constexpr int NT = DUAL ? 128 : 256, KEYS = BN / NU;
                for (int hf = 0; hf < NU && ok; ++hf) {
                    const int u = tt * NU + hf;
                    ok = sleep_wait(&bars[Y::B_FULL + u % NS], (u / NS) & 1, abort, err);
                    if (!ok) break;
                    const int from = max(0, tail - hf * KEYS);
                    uint8_t *vt = smem + Y::KV_OFF + (u % NS) * Y::UNIT;
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
            warp_arrive(&bars[Y::B_P + (DUAL ? x : (j & 1))]);
        }
        // ---- output rows
        if (ok && nb > 0)
            ok = DUAL ? sleep_wait(&bars[Y::B_O + x], 0, abort, err)
                      : sleep_wait(&bars[Y::B_O], (nb - 1) & 1, abort, err);
        if constexpr (!DUAL) {
            if (ok && nb > 0) {
                float *rb = red + (wphase & 1) * 256;
                rb[wg * 128 + r] = l;
                warp_arrive(&bars[Y::B_WG]);
                ok = sleep_wait(&bars[Y::B_WG], wphase & 1, abort, err);
                if (ok) l = wg == 0 ? l + rb[128 + r] : rb[r] + l;
            }
        }
        tc_fence_after();
        const bool nan_row = !ok || sq.lk < 0;
        const float inv = nan_row ? NaN : l == 0.f ? 0.f : 1.f / l;
        const size_t row = (size_t)(sq.q0 + t0 + ti) * P.Hq + h;
        if (live && P.lse != nullptr && (DUAL || wg == 0))
            P.lse[row] = nan_row ? NaN : l == 0.f ? -INFINITY : m * P.softmax_scale + logf(l);
#pragma unroll
        for (int i = 0; i < OC / 32; ++i) {
            float o[32];
            if (nb > 0) {
                tmem_ld32_nowait(tO + 32u * i, o);
                tmem_wait32(o);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = (nb > 0 && l != 0.f) ? o[e] * inv : (nan_row ? NaN : 0.f);
            if (live) {
            const size_t e0 = row * D + (DUAL ? 0 : 128 * wg) + 32 * i;
            if (P.out_dtype == PA_F32) {
                float4 *d = reinterpret_cast<float4 *>(reinterpret_cast<float *>(P.out) + e0);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            } else {
                uint4 *d = reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(P.out) + e0);
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    w[e] = P.out_dtype == PA_BF16 ? pack_bf16x2(o[2 * e], o[2 * e + 1])
                                                  : pack_f16x2(o[2 * e], o[2 * e + 1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) d[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            }
            }
            __syncwarp();
        }
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
                          unsigned ctas, cudaStream_t s) {
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
    const long long ctas = ((long long)p->total_q / tq_tokens + std::min(p->num_seqs, p->total_q)) * p->num_kv_heads;
    if (ctas > 0x7FFFFFFFll) return PA_ERR_UNSUPPORTED;
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
    P.out_dtype = p->out_dtype;
    P.causal = p->causal;
    P.softmax_scale = p->softmax_scale;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    const bool bf = p->dtype == PA_BF16;
    switch (D) {
        case 64: e = bf ? pa::prompt::launch_prompt<64, true>(tq, tk, tv, P, (unsigned)ctas, s)
                        : pa::prompt::launch_prompt<64, false>(tq, tk, tv, P, (unsigned)ctas, s); break;
        case 128: e = bf ? pa::prompt::launch_prompt<128, true>(tq, tk, tv, P, (unsigned)ctas, s)
                         : pa::prompt::launch_prompt<128, false>(tq, tk, tv, P, (unsigned)ctas, s); break;
        default: e = bf ? pa::prompt::launch_prompt<256, true>(tq, tk, tv, P, (unsigned)ctas, s)
                        : pa::prompt::launch_prompt<256, false>(tq, tk, tv, P, (unsigned)ctas, s); break;
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
