// Accumulated attention weight for many query rows per kv head, on the
// fifth-generation tensor cores.
//
//   S^T = K q^T   M = 128 tokens, N = up to 256 rows, K = head dim (once per
//                 term of the queries), f16 or bf16
//   mass[t] += sum over rows of exp(c S^T[t, r] - lse_r)   t < vis_r
//
// The warp-level kernel (pa_mass.cu) keeps the query in registers, which
// holds up to 16 rows; its operand traffic bounds it there and beyond.  Here a tile of 128
// tokens is one A operand in shared memory, the rows are one B operand beside
// it, and the sum over rows needs no shuffles: in tensor memory a token is a
// lane, so one thread adds up its token's rows.
//
// Measured on a GB300: 32 causal rows of 64 / 8 heads (256 rows per kv head) over
// 16 requests of 2048-16384 tokens, INT8 head dim 128 with per-channel scales
// 173 us; the two-term products alone are 92 us at the measured bf16 rate, the
// sums (one ex2 per row and token) and the decoding run beside them, and each new
// (request, kv head) costs the pipeline its staging of the query rows, some 6 us
// (256 rows; 20 us, and 251 us in all, when their terms were packed row by row).
// The warp-level kernel takes 7.2 ms for the same call; where the border between
// the two lies, and what they measure there, stands at the entry point beside it.
//
// Roles (17 warps at work): two loader warpgroups take alternate tiles -- 16-bit
// codes are copied asynchronously into the swizzled operand layout, quantized
// ones loaded one to four tiles ahead into registers, decoded exactly and stored there;
// one warp issues the MMAs; two epilogue warpgroups, one per S^T buffer, sum and
// update the total (a tile always falls to the same warpgroup, so the passes
// over chunks of rows are ordered) and stage the query rows of each segment.
// Tiles in logical order (request, kv head, tile) are shared evenly by
// persistent CTAs.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "pa_mass.cuh"
#include "pa_tc_warp.cuh"

namespace pa {
namespace mass {

namespace mtc {

using namespace tc;

constexpr int CH = 128;                                   // tokens per tile
constexpr int W_EPI = 8, W_MMA = 16;   // warps 0-7 load, 8-15 sum, 16 issues (17-19 idle: their registers go to the others)
constexpr int THREADS = 640;
constexpr int REGS_LAUNCH = 96, REGS_WORK = 104, REGS_MMA = 64;
static_assert(512 * REGS_WORK + 128 * REGS_MMA <= THREADS * REGS_LAUNCH, "register split exceeds the launch");

template <int D>
struct Lay {
    static constexpr int NA = D == 64 ? 8 : D == 128 ? 6 : 3;  // A buffers at most
    static constexpr int RMAX = D == 256 ? 128 : 256;          // query rows of a chunk
    static constexpr int A_BYTES = CH * D * 2;
    static constexpr int CST_OFF = 0;                          // [2 segments][RMAX / 2 pairs] {sc0, sc1, -lse0, -lse1}
    static constexpr int VIS_OFF = CST_OFF + 2 * (RMAX / 2) * 16;  // [2][RMAX]
    static constexpr int BAR_OFF = VIS_OFF + 2 * RMAX * 4;
    enum {
        B_AFULL = 0,              // [NA] tile in place
        B_AFREE = B_AFULL + NA,   // [NA] its MMAs complete
        B_SFULL = B_AFREE + NA,   // [2]
        B_SFREE = B_SFULL + 2,    // [2]
        B_QFULL = B_SFREE + 2,    // query rows of the segment staged
        B_QFREE = B_QFULL + 1,    // MMAs of the segment complete
        B_DONE = B_QFREE + 1,
        NBARS = B_DONE + 1
    };
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;  // [0] tmem, [1] abort, [2] errors, [4 ..] scan
    static constexpr int A_OFF = (MISC_OFF + 128 + 1023) / 1024 * 1024;
    // then the A buffers, the query operand and the prefix sums (B + 1 ints)
    static constexpr int ROOM = 227 * 1024 - A_OFF - (MAX_B + 1) * 4;
};

// the CTA's tiles: pieces of one (request, kv head), each walked once per chunk of rows
struct Walk {
    int b, g, u, ua, ue, c, L;  // tile u of ua .. ue - 1, chunk c
    long long x, x1;            // next piece's position, end of the share
    bool end;
};

__device__ __forceinline__ void walk_piece(Walk &w, const MassParams &P, const int *ps) {
    if (w.x >= w.x1) {
        w.end = true;
        return;
    }
    w.b = request_of(ps, P.B, (int)(w.x / P.Hkv));
    const int units = ps[w.b + 1] - ps[w.b];
    const long long rem = w.x - (long long)ps[w.b] * P.Hkv;
    w.g = (int)(rem / units);
    w.ua = w.u = (int)(rem % units);
    w.ue = (int)min((long long)units, w.ua + (w.x1 - w.x));
    w.x += w.ue - w.ua;
    w.c = 0;
    w.L = P.context_lens[w.b];
}

__device__ __forceinline__ void walk_next(Walk &w, const MassParams &P, const int *ps, int chunks) {
    if (++w.u < w.ue) return;
    if (++w.c < chunks) w.u = w.ua;
    else walk_piece(w, P, ps);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// byte offset of 16-byte chunk c of operand row t, rows `rows` of 128-byte panels
__device__ __forceinline__ uint32_t op_off(int rows, int t, int c) {
    return (uint32_t)((c >> 3) * rows * 128 + t * 128 + (((c & 7) ^ (t & 7)) << 4));
}

// the sum over rows of a tile that some row does not see all of (the last
// ones of a request): rows taken two by two, each against its visible length
__device__ __noinline__ float masked_sum(uint32_t tl, int rp, const float *cst, const int *vs, int tok, float ts) {
    float tot = 0.f;
#pragma unroll 1
    for (int r0 = 0; r0 < rp; r0 += 8) {
        uint32_t z[8];
        tmem_ld8_nowait(tl + (uint32_t)r0, z);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float d = __uint_as_float(z[e]);
            const int r = r0 + e;
            d = fmaf(d * ts, cst[(r >> 1) * 4 + (r & 1)], cst[(r >> 1) * 4 + 2 + (r & 1)]);
            if (tok < vs[r]) tot += ex2(d);
        }
    }
    return tot;
}

}  // namespace mtc

template <int D, int KV>
__global__ void __launch_bounds__(mtc::THREADS, 1) pa_mass_tc_kernel(MassParams P, int nt, int rows_c, int chunks, int na) {
    using namespace mtc;
    using Y = Lay<D>;
    constexpr int BITS = KV == PA_INT4 ? 4 : (KV == PA_E4M3 || KV == PA_INT8) ? 8 : 16;
    constexpr bool BF = KV == PA_BF16;
    const int NA = na, q_off = Y::A_OFF + na * Y::A_BYTES;  // A buffers; the query operand behind them
    constexpr int RB = D * BITS / 8, PR = RB / 16;  // bytes and 16-byte pieces per token
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Y::BAR_OFF);
    int *misc = reinterpret_cast<int *>(smem + Y::MISC_OFF);
    volatile int *abort = misc + 1;
    int *ps = reinterpret_cast<int *>(smem + q_off + nt * rows_c * D * 2);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const float NaN = __int_as_float(0x7fc00000);
    if (sb & 1023) {
        if (tid == 0 && P.dev_error) atomicOr(P.dev_error, PA_DEV_ERR_TIMEOUT);
        return;
    }
    grid_dependents_launch();
    grid_dependency_wait();
    const bool bad_len = scan_units<THREADS, CH>(P, ps, misc + 4);
    if (bad_len && blockIdx.x == 0 && P.dev_error) atomicOr(P.dev_error, PA_DEV_ERR_CONTEXT_LEN);
    const long long N = (long long)ps[P.B] * P.Hkv;
    const long long x0 = blockIdx.x * N / gridDim.x, x1 = (blockIdx.x + 1) * N / gridDim.x;
    if (x0 >= x1) return;

    if (tid == 0) {
        for (int i = 0; i < Y::NBARS; ++i) {
            uint32_t c = 1;
            if ((i >= Y::B_AFULL && i < Y::B_AFULL + Y::NA) || (i >= Y::B_SFREE && i < Y::B_SFREE + 2)) c = 4;
            if (i == Y::B_QFULL) c = 8;
            mbar_init(&bars[i], c);
        }
        misc[1] = 0;
        misc[2] = 0;
        mbar_fence_init();
    }
    if (warp == W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sb + Y::MISC_OFF)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform(misc[0]);
    uint32_t err = 0;
    Walk w;
    w.x = x0;
    w.x1 = x1;
    w.end = false;
    walk_piece(w, P, ps);

    if (warp < W_EPI) {
        regs_inc<REGS_WORK>();
        // ================================================== loaders: tile i by warpgroup i & 1
        const int wg = warp >> 2, wq = warp & 3;  // the warp's 32 tokens: 32 wq ..
        long long i = wg;                         // the next tile to publish
        struct Slot {
            int slot, par;  // buffer, parity of its uses
        };
        Slot put = {wg, 0};
        auto two_on = [&](Slot a) -> Slot {
            Slot b;
            const bool wrap = a.slot + 2 >= NA;
            b.slot = wrap ? a.slot + 2 - NA : a.slot + 2;
            b.par = a.par ^ (wrap ? 1 : 0);
            return b;
        };
        // The warp's 32 tokens are two runs of 16 rows, each contiguous in its
        // block.  Their places are known QD tiles of this warpgroup ahead, so that
        // the block ids have arrived when the rows are asked for.
        struct Place {
            int id[2], off[2], left;  // blocks, byte offsets in them, tokens of the 32 that exist
        };
        constexpr int QD = 2;
        Place pl[QD];
        auto step = [&]() {
            if (!w.end) walk_next(w, P, ps, chunks);
        };
        auto place = [&](Place &q) {
            q.left = w.end ? 0 : w.L - (w.u * CH + 32 * wq);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = w.u * CH + 32 * wq + 16 * h;
                const int col = (int)__umulhi((unsigned)t, P.bs_mul);
                q.id[h] = (!w.end && t < w.L) ? P.block_table[(size_t)w.b * P.tbl + col] : 0;
                q.off[h] = (w.g * P.bs + t - col * P.bs) * RB;
            }
            step();
            step();
        };
        if (wg == 1) step();
#pragma unroll
        for (int q = 0; q < QD; ++q) place(pl[q]);
        auto rotate = [&]() {
#pragma unroll
            for (int q = 0; q + 1 < QD; ++q) pl[q] = pl[q + 1];
            place(pl[QD - 1]);
        };
        const long long mine = (x1 - x0) * chunks;  // tiles of the CTA, all passes
#ifdef PA_FAULT_INJECT
        // tile (word >> 8) - 1 of CTA 0 is never published
        const int fi = P.dev_error && blockIdx.x == 0 ? (int)(*P.dev_error >> 8) - 1 : -1;
#else
        constexpr int fi = -1;
#endif
        const uint8_t *run[2];
        auto runs_of = [&](const Place &q) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                run[h] = q.id[h] >= 1 && q.id[h] < P.num_blocks ? P.k_pool + (size_t)q.id[h] * P.k_block + q.off[h]
                                                               : nullptr;
        };
        // Piece k (of PR) of this lane: piece pq of the warp's token k TK + tq, in run
        // k / (PR / 2).  A piece becomes OC operand chunks; eight lanes side by side
        // hold one panel of OC tokens, so that what they store at a time falls into
        // eight different chunk positions of the swizzle (lanes along a row would
        // meet two and four at a time).
        constexpr int OC = 16 / BITS, LP = 8 / OC, TK = 32 / PR;
        const int tq = (lane >> 3) / (D / 64) * OC + (lane & 7) / LP;
        const int pq = (lane >> 3) % (D / 64) * LP + (lane & 7) % LP;
        auto piece = [&](int k, int left, bool &live) -> const uint8_t * {
            const int h = k < PR / 2 ? 0 : 1;
            live = run[h] != nullptr && k * TK + tq < left;
            return live ? run[h] + ((k * TK + tq - h * 16) * PR + pq) * 16 : P.k_pool;
        };
        if constexpr (BITS == 16) {
            // Up to PF tiles of this warpgroup in flight, then publish the oldest.  With
            // a buffer or two to spare beside the two warpgroups' tiles none waits for
            // the other's tile before it publishes its own (16 x 2048-16384 f16 tokens,
            // head dim 128, 96 rows, five buffers: 71 us with two each, 104 with three;
            // 32 rows, six buffers: 72 with two each, 82 with three).
            const int PF = NA < 4 ? 1 : (NA - 1) / 2;
            long long ai = wg;    // the next tile to copy
            Slot at = {wg, 0};    // its buffer
            while (i < mine) {
                if (ai < mine && ai - i < 2 * PF) {
                    if (ai >= NA && !sleep_wait(&bars[Y::B_AFREE + at.slot], at.par ^ 1, abort, err)) break;
                    const uint32_t dst = sb + Y::A_OFF + at.slot * Y::A_BYTES;
                    const int left = pl[0].left;
                    runs_of(pl[0]);
#pragma unroll 4
                    for (int k = 0; k < PR; ++k) {
                        bool live;
                        const uint8_t *src = piece(k, left, live);
                        cp_async16(dst + op_off(CH, 32 * wq + k * TK + tq, pq), src, live);
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    ai += 2;
                    at = two_on(at);
                    rotate();
                    if (ai < mine && ai - i < 2 * PF) continue;
                }
                const long long newer = (ai - i) / 2 - 1;  // copies that may stay in flight
                if (newer == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
                else if (newer == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
                else asm volatile("cp.async.wait_group 0;" ::: "memory");
                fence_proxy_async_smem();
                if (i != fi) warp_arrive(&bars[Y::B_AFULL + put.slot]);
                put = two_on(put);
                i += 2;
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        } else {
            // The next PF tiles of this warpgroup are on their way in registers, 64 of
            // them whatever a row's size: with one tile of 8 pieces ahead the loads'
            // latency bounds few rows (24 rows INT8 head dim 128: 66 us).
            constexpr int PF = PR >= 16 ? 1 : 16 / PR;
            uint4 raw[PF][PR];
            auto fetch = [&](uint4 *to) {
                const int left = pl[0].left;
                runs_of(pl[0]);
#pragma unroll
                for (int k = 0; k < PR; ++k) {
                    bool live;
                    const uint8_t *src = piece(k, left, live);
                    to[k] = live ? __ldg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0u, 0u, 0u, 0u);
                }
            };
#pragma unroll
            for (int p = 0; p < PF; ++p) {
                if (p > 0) rotate();
                fetch(raw[p]);
            }
            bool go = true;
            while (go && i < mine) {
#pragma unroll
                for (int p = 0; p < PF; ++p) {
                    if (!go || i >= mine) break;
                    const int slot = put.slot;
                    if (i >= NA && !sleep_wait(&bars[Y::B_AFREE + slot], put.par ^ 1, abort, err)) {
                        go = false;
                        break;
                    }
                    uint8_t *dst = smem + Y::A_OFF + slot * Y::A_BYTES;
#pragma unroll
                    for (int k = 0; k < PR; ++k) {
                        uint32_t wd[4 * OC];
                        decode<KV>(raw[p][k], wd);
#pragma unroll
                        for (int o = 0; o < OC; ++o)
                            *reinterpret_cast<uint4 *>(dst + op_off(CH, 32 * wq + k * TK + tq, pq * OC + o)) =
                                make_uint4(wd[4 * o], wd[4 * o + 1], wd[4 * o + 2], wd[4 * o + 3]);
                    }
                    fence_proxy_async_smem();
                    if (i != fi) warp_arrive(&bars[Y::B_AFULL + slot]);
                    rotate();
                    fetch(raw[p]);
                    i += 2;
                    put = two_on(put);
                }
            }
        }
    } else if (warp < W_MMA) {
        regs_inc<REGS_WORK>();
        // ================================================== sums over rows; query staging
        const int wg = (warp - W_EPI) >> 2, qd = warp & 3;
        const int t = 32 * qd + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16) + 256u * wg;
        const int rp = rows_c;  // rows of the B operand
        int seg = -1, sphase = 0;
        bool ok = true;
        int f_blk = 0;
        float f_old = 0.f;
        for (; !w.end && ok; walk_piece(w, P, ps)) {
            const int u1 = w.ua + ((w.ua ^ wg) & 1);  // this warpgroup's first tile of the piece
            const int32_t *table = P.block_table + (size_t)w.b * P.tbl;
            float *mass = P.mass + ((size_t)w.b * P.Hkv + w.g) * P.max_ctx;
            for (w.c = 0; w.c < chunks && ok; ++w.c) {
                const float dec = w.c == 0 ? P.decay : 1.f;
                // the thread's token of tile u: its block and its total so far (of
                // the passes before this one, which this thread wrote)
                auto fetch_token = [&](int u) {
                    const int tok = u * CH + t;
                    const bool in = u < w.ue && tok < w.L;
                    f_blk = in ? table[__umulhi((unsigned)tok, P.bs_mul)] : 0;
                    f_old = in && dec != 0.f ? mass[tok] : 0.f;
                };
                fetch_token(u1);
                // ---- a new segment: its query rows
                ++seg;
                float *cst = reinterpret_cast<float *>(smem + Y::CST_OFF) + (seg & 1) * (Y::RMAX / 2) * 4;
                int *vs = reinterpret_cast<int *>(smem + Y::VIS_OFF) + (seg & 1) * Y::RMAX;
                const float *fold = P.k_mode == PA_SCALE_CHANNEL ? P.k_scale + (size_t)w.g * D : nullptr;
                const float ks = P.k_mode == PA_SCALE_TENSOR ? P.k_scale[0] : 1.f;
                const bool scaled = !BF && (fold != nullptr || P.q_dtype == PA_BF16);
                constexpr int WP = 64 / BITS;  // operand words per raw piece
                float2 fv[D / 64];
#pragma unroll
                for (int k = 0; k < D / 64; ++k) {
                    const int pc = (lane + 32 * k) / WP, wd = (lane + 32 * k) % WP;
                    fv[k] = fold ? make_float2(fold[channel_of<BITS>(pc, wd, 0)], fold[channel_of<BITS>(pc, wd, 1)])
                                 : make_float2(1.f, 1.f);
                }
                // A warp takes QB rows at a time: all their loads in flight together,
                // and those of its next ones while these are stored.
                constexpr int QB = D == 256 ? 4 : 8, KW = D / 64;
                uint32_t raw[QB][KW];  // lane: operand words lane, lane + 32, ... (pairs of channels)
                float lse;
                int vis;
                auto load_rows = [&](int rr0) {
                    // lane i holds the statistics of row i: one load for all of them (a load
                    // per row into one register would wait for the row before)
                    lse = -INFINITY;
                    vis = 0x7FFFFFFF;  // rows past R never count, and do not force the masked sum either
                    const int lr = w.c * rows_c + rr0 + lane;
                    if (lane < QB && rr0 + lane < rows_c && lr < P.R) {
                        const int lj = lr / P.G;
                        lse = P.lse[((size_t)w.b * P.n + lj) * P.Hq + w.g * P.G + (lr - lj * P.G)];
                        vis = P.causal ? w.L - (P.n - 1 - lj) : w.L;
                    }
                    int r = w.c * rows_c + rr0, j = r / P.G, hg = r - j * P.G;
#pragma unroll
                    for (int i = 0; i < QB; ++i, ++r) {
                        const bool rok = rr0 + i < rows_c && r < P.R;
                        const size_t row = ((size_t)w.b * P.n + j) * P.Hq + w.g * P.G + hg;
                        const uint16_t *src = reinterpret_cast<const uint16_t *>(P.q + row * (2 * D));
#pragma unroll
                        for (int k = 0; k < KW; ++k) {
                            if constexpr (BITS == 4) {
                                const int c0 = channel_of<4>((lane + 32 * k) / WP, (lane + 32 * k) % WP, 0);
                                raw[i][k] = rok ? (uint32_t)src[c0] | ((uint32_t)src[c0 + 4] << 16) : 0u;
                            } else {
                                raw[i][k] = rok ? reinterpret_cast<const uint32_t *>(src)[lane + 32 * k] : 0u;
                            }
                        }
                        if (++hg == P.G) {
                            hg = 0;
                            ++j;
                        }
                    }
                };
                int rr0 = (warp - W_EPI) * QB;
                if (rr0 < rp) load_rows(rr0);
                if (seg > 0 && !sleep_wait(&bars[Y::B_QFREE], (seg - 1) & 1, abort, err)) {
                    ok = false;
                    break;
                }
                for (; rr0 < rp; rr0 += 8 * QB) {
                    float2 v[QB][KW];
#pragma unroll
                    for (int i = 0; i < QB; ++i)
#pragma unroll
                        for (int k = 0; k < KW; ++k) {
                            const uint32_t x = raw[i][k];
                            float2 f = P.q_dtype == PA_BF16
                                           ? make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u))
                                           : __half22float2(*reinterpret_cast<const __half2 *>(&x));
                            f.x *= fv[k].x;
                            f.y *= fv[k].y;
                            v[i][k] = f;
                        }
                    const float my_lse = lse;
                    const int my_vis = vis;
                    if (rr0 + 8 * QB < rp) load_rows(rr0 + 8 * QB);
                    float my_down = 1.f;
                    if (scaled) {
                        float mx[QB];
#pragma unroll
                        for (int i = 0; i < QB; ++i) {
                            mx[i] = 0.f;
#pragma unroll
                            for (int k = 0; k < KW; ++k)
                                mx[i] = fmaxf(mx[i], fmaxf(fabsf(v[i][k].x), fabsf(v[i][k].y)));
                        }
#pragma unroll
                        for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
                            for (int i = 0; i < QB; ++i) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
#pragma unroll
                        for (int i = 0; i < QB; ++i) {
                            int ex = 0;
                            if (mx[i] > 0.f && mx[i] < 3.0e38f) ex = (int)(__float_as_uint(mx[i]) >> 23) - 126;
                            ex = max(-120, min(120, ex));
                            const float up = __int_as_float((127 - ex) << 23);
                            if (lane == i) my_down = __int_as_float((127 + ex) << 23);
#pragma unroll
                            for (int k = 0; k < KW; ++k) {
                                v[i][k].x *= up;
                                v[i][k].y *= up;
                            }
                        }
                    }
                    // term by term, the words of all rows beside one another: word lane + 32 k
                    // of a row is in 16-byte chunk lane / 4 of channel panel k
                    uint8_t *dst = smem + q_off + rr0 * 128 + 4 * (lane & 3);
#pragma unroll 1
                    for (int q = 0; q < nt; ++q, dst += rp * D * 2) {
#pragma unroll
                        for (int i = 0; i < QB; ++i)
#pragma unroll
                            for (int k = 0; k < KW; ++k) {
                                float2 &f = v[i][k];
                                const uint32_t x = pack2<BF>(f.x, f.y);
                                *reinterpret_cast<uint32_t *>(dst + k * rp * 128 + i * 128 +
                                                              (((lane >> 2) ^ ((rr0 + i) & 7)) << 4)) = x;
                                if constexpr (BF) {
                                    f.x -= __uint_as_float(x << 16);
                                    f.y -= __uint_as_float(x & 0xFFFF0000u);
                                } else {
                                    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&x));
                                    f.x -= h.x;
                                    f.y -= h.y;
                                }
                            }
                    }
                    if (lane < QB) {
                        const int rr = rr0 + lane;
                        const bool on = my_lse != -INFINITY;
                        // in the exp2 domain: the two roundings by log2 e cost some 2^-24 of a
                        // score or of lse, as much as fp32 scores have anyway
                        cst[(rr >> 1) * 4 + (rr & 1)] = on ? P.softmax_scale * ks * my_down * LOG2E : 0.f;
                        cst[(rr >> 1) * 4 + 2 + (rr & 1)] = on ? -my_lse * LOG2E : -INFINITY;
                        vs[rr] = (my_vis != 0x7FFFFFFF && !on) ? 0 : my_vis;
                    }
                }
                fence_proxy_async_smem();
                warp_arrive(&bars[Y::B_QFULL]);
                if (!sleep_wait(&bars[Y::B_QFULL], seg & 1, abort, err)) {
                    ok = false;
                    break;
                }
                int mn = 0x7FFFFFFF;
                for (int r = lane; r < rp; r += 32) mn = min(mn, vs[r]);
                const bool seg_off = __any_sync(0xffffffffu, mn <= 0);
                const ulonglong2 *cst2 = reinterpret_cast<const ulonglong2 *>(cst);
                // ---- its tiles
                for (int u = u1; u < w.ue; u += 2) {
                    const int tok = u * CH + t;
                    const bool in = tok < w.L, okb = f_blk >= 1 && f_blk < P.num_blocks;
                    const float old = f_old;
                    float ts = 1.f;
                    if (KV == PA_E4M3 && P.k_mode == PA_SCALE_TOKEN && in && okb)
                        ts = __ldg(reinterpret_cast<const float *>(P.k_pool + (size_t)f_blk * P.k_block + P.k_codes) +
                                   (size_t)w.g * P.bs + tok % P.bs);
                    fetch_token(u + 2);
                    // some row may not see some token of the tile (or saw nothing at all: lse = -inf)
                    const bool masked = seg_off || u * CH + CH > w.L - P.n;
                    ok = sleep_wait(&bars[Y::B_SFULL + wg], sphase & 1, abort, err);
                    if (!ok) break;
                    ++sphase;
                    tc_fence_after();
                    const uint64_t ts2 = f2(ts, ts);
                    uint64_t tot[2] = {0, 0};
                    auto add_rows = [&](auto ncol, int r0) {
                        constexpr int C = decltype(ncol)::value;
                        float z[C];
                        if constexpr (C == 32) {
                            tmem_ld32_nowait(tl + (uint32_t)r0, z);
                            tmem_wait32(z);
                        } else {
                            tmem_ld16_nowait(tl + (uint32_t)r0, reinterpret_cast<uint32_t *>(z));
                            tmem_wait16(z);
                        }
#pragma unroll
                        for (int e = 0; e < C; e += 2) {
                            const ulonglong2 c = cst2[(r0 + e) >> 1];  // {scales, -lse} of two rows
                            uint64_t d = f2(z[e], z[e + 1]);
                            if (KV == PA_E4M3) d = mul2(d, ts2);
                            d = fma2(d, c.x, c.y);
                            float a, b;
                            f2_split(d, a, b);
                            tot[(e >> 1) & 1] = add2(tot[(e >> 1) & 1], f2(ex2(a), ex2(b)));
                        }
                    };
                    float got = 0.f;
                    if (masked) {
                        got = masked_sum(tl, rp, cst, vs, tok, ts);
                    } else {
                        int r0 = 0;
#pragma unroll 1
                        for (; r0 + 32 <= rp; r0 += 32) add_rows(std::integral_constant<int, 32>(), r0);
                        if (r0 < rp) add_rows(std::integral_constant<int, 16>(), r0);
                        float a, b;
                        f2_split(add2(tot[0], tot[1]), a, b);
                        got = a + b;
                    }
                    tc_fence_before();
                    warp_arrive(&bars[Y::B_SFREE + wg]);
                    if (in) {
                        mass[tok] = !okb ? NaN : dec != 0.f ? fmaf(dec, old, got) : got;
                        if (!okb) err |= PA_DEV_ERR_BLOCK_ID;
                    }
                }
            }
            if (!ok) break;
        }
        if (!ok) {  // a wait ran out: the tiles of the whole share are NaN
            w.x = x0;
            w.end = false;
            for (walk_piece(w, P, ps); !w.end; walk_piece(w, P, ps))
                for (int u = w.ua + ((w.ua ^ wg) & 1); u < w.ue; u += 2)
                    if (u * CH + t < w.L) P.mass[((size_t)w.b * P.Hkv + w.g) * P.max_ctx + u * CH + t] = NaN;
        }
    } else {
        regs_dec<REGS_MMA>();
        // ================================================== MMA issue (one warp)
        if (warp == W_MMA) {
            const uint64_t qpanel = (uint64_t)(rows_c * 128 >> 4);  // descriptor step between channel panels of the rows
            constexpr uint32_t FMT = BF ? (1u << 7) | (1u << 10) : 0u;
            const uint32_t id = idesc(CH, rows_c, 0) | FMT;
            const uint64_t ad = sdesc(sb + Y::A_OFF, 16, 1024, 2), qd = sdesc(sb + q_off, 16, 1024, 2);
            int slot = 0, spar = 0, seg = 0;
            uint32_t used = 0, bpar = 0;  // per S buffer: whether it was used, parity of its uses
            bool ok = true;
            for (; !w.end && ok; walk_piece(w, P, ps)) {
                const int ua = uniform(w.ua), ue = uniform(w.ue);
                for (int c = 0; c < chunks && ok; ++c, ++seg) {
                    ok = sleep_wait(&bars[Y::B_QFULL], seg & 1, abort, err);
                    for (int u = ua; u < ue && ok; ++u) {
                        const int buf = u & 1;
                        ok = sleep_wait(&bars[Y::B_AFULL + slot], spar, abort, err);
                        // (the use before: one parity back)
                        if (ok && ((used >> buf) & 1))
                            ok = sleep_wait(&bars[Y::B_SFREE + buf], ((bpar >> buf) & 1) ^ 1, abort, err);
                        if (!ok) break;
                        used |= 1u << buf;
                        bpar ^= 1u << buf;
                        tc_fence_after();
                        const uint64_t a = ad + (uint32_t)(slot * (Y::A_BYTES >> 4));
                        uint64_t q = qd;
                        const uint32_t d = tmem + 256u * buf;
                        // the terms of a query one after the other, into the same sums
                        for (int t = 0; t < nt; ++t)
#pragma unroll
                            for (int pn = 0; pn < D / 64; ++pn, q += qpanel)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_f16_w(d, a + (uint32_t)((pn * CH * 128 + 32 * k) >> 4), q + 2u * k, id,
                                              (t > 0 || pn > 0 || k > 0) ? 1u : 0u);
                        mma_commit_w(&bars[Y::B_SFULL + buf]);
                        mma_commit_w(&bars[Y::B_AFREE + slot]);
                        const bool wrap = slot == NA - 1;
                        slot = wrap ? 0 : slot + 1;
                        spar ^= wrap ? 1 : 0;
                    }
                    if (ok) mma_commit_w(&bars[Y::B_QFREE]);
                }
            }
            mma_commit_w(&bars[Y::B_DONE]);
            if (lane == 0) (void)mbar_wait_bounded(&bars[Y::B_DONE], 0, nullptr);
        }
        __syncwarp();
    }

    if (err) atomicOr(reinterpret_cast<unsigned *>(misc + 2), err);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W_MMA) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    if (tid == 0 && misc[2] != 0 && P.dev_error) atomicOr(P.dev_error, (uint32_t)misc[2]);
}

template <int D, int KV>
cudaError_t launch_tc(const MassParams &P, int nt, int sms, cudaStream_t s) {
    using Y = mtc::Lay<D>;
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev >= 64 || !(done.load(std::memory_order_relaxed) & bit)) {
        // the register split draws on what the block was launched with
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, pa_mass_tc_kernel<D, KV>);
        if (e != cudaSuccess) return e;
        if (at.numRegs < mtc::REGS_LAUNCH) return cudaErrorLaunchOutOfResources;
        e = cudaFuncSetAttribute(pa_mass_tc_kernel<D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    // chunks of rows of equal size, as few as fit the operand beside two A buffers; then as many A buffers as fit
    const int row_bytes = D * 2 * nt;
    const int most = std::min((int)Y::RMAX, (Y::ROOM - 2 * Y::A_BYTES) / row_bytes / 16 * 16);
    int chunks = (P.R + most - 1) / most;
    // (multiples of the MMA's N step)
    const int rows_c = ((P.R + chunks - 1) / chunks + 15) / 16 * 16;
    chunks = (P.R + rows_c - 1) / rows_c;
    const int na = std::min((int)Y::NA, (Y::ROOM - rows_c * row_bytes) / Y::A_BYTES);
    const int smem = Y::A_OFF + na * Y::A_BYTES + rows_c * row_bytes + (P.B + 1) * 4;
    // no CTA without a tile of the longest possible batch
    const long long tiles = (long long)P.B * P.Hkv * ((P.max_ctx + mtc::CH - 1) / mtc::CH);
    const int ctas = (int)std::max(1ll, std::min<long long>(sms, tiles));
    return launch_pdl(pa_mass_tc_kernel<D, KV>, dim3(ctas), dim3(mtc::THREADS), (size_t)smem, s, P, nt, rows_c, chunks, na);
}

template <int D>
cudaError_t dispatch_tc(const MassParams &P, int kv, int nt, int sms, cudaStream_t s) {
    switch (kv) {
        case PA_F16: return launch_tc<D, PA_F16>(P, nt, sms, s);
        case PA_BF16: return launch_tc<D, PA_BF16>(P, nt, sms, s);
        case PA_E4M3: return launch_tc<D, PA_E4M3>(P, nt, sms, s);
        case PA_INT8: return launch_tc<D, PA_INT8>(P, nt, sms, s);
        case PA_INT4:
            if constexpr (D >= 128) return launch_tc<D, PA_INT4>(P, nt, sms, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_mass_tc(const MassParams &P, int kv, int D, int nt, int sms, cudaStream_t s) {
    return D == 64 ? dispatch_tc<64>(P, kv, nt, sms, s) : D == 128 ? dispatch_tc<128>(P, kv, nt, sms, s)
                                                                   : dispatch_tc<256>(P, kv, nt, sms, s);
}

}  // namespace mass
}  // namespace pa
