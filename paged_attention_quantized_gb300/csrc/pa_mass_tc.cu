// Accumulated attention weight for many query rows per kv head, on the
// fifth-generation tensor cores.
//
//   S^T = K q^T   M = 128 tokens, N = rows (times two for two-term queries),
//                 K = head dim, f16 or bf16
//   mass[t] += sum over rows of exp(c S^T[t, r] - lse_r)   t < vis_r
//
// The warp-level kernel (pa_mass.cu) keeps the query in registers, which
// holds up to 16 rows; beyond that its operand traffic bounds it.  Here a tile of 128
// tokens is one A operand in shared memory, the rows are one B operand beside
// it, and the sum over rows needs no shuffles: in tensor memory a token is a
// lane, so one thread adds up its token's rows.
//
// Roles (17 warps): two loader warpgroups take alternate tiles -- 16-bit codes
// are copied asynchronously into the swizzled operand layout, quantized ones
// loaded a tile ahead into registers, decoded exactly and stored there; one
// warp issues the MMAs; two epilogue warpgroups, one per S^T buffer, sum and
// update the total (a tile always falls to the same warpgroup, so the passes
// over chunks of rows are ordered) and stage the query rows of each segment.
// Tiles in logical order (request, kv head, tile) are shared evenly by
// persistent CTAs.
#include <algorithm>
#include <atomic>

#include "pa_mass.cuh"
#include "pa_tc.cuh"

namespace pa {
namespace mass {

namespace mtc {

using namespace tc;

constexpr int CH = 128;                                   // tokens per tile
constexpr int W_EPI = 8, W_MMA = 16, THREADS = 17 * 32;  // warps 0-7 load

template <int D>
struct Lay {
    static constexpr int NA = D == 64 ? 4 : D == 128 ? 3 : 2;  // A buffers
    static constexpr int NMAX = D == 256 ? 128 : 256;          // rows of the B operand (terms included)
    static constexpr int PANELS = D / 64;
    static constexpr int A_BYTES = CH * D * 2;
    static constexpr int A_OFF = 0;
    static constexpr int Q_OFF = NA * A_BYTES;
    static constexpr int Q_BYTES = NMAX * D * 2;
    static constexpr int CST_OFF = Q_OFF + Q_BYTES;            // [2 segments][128 pairs] {sc0, sc1, -ls0, -ls1}
    static constexpr int VIS_OFF = CST_OFF + 2 * (NMAX / 2) * 16;  // [2][NMAX]
    static constexpr int BAR_OFF = VIS_OFF + 2 * NMAX * 4;
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
    static constexpr int PS_OFF = MISC_OFF + 128;         // prefix sums (B + 1 ints)
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

}  // namespace mtc

template <int D, int KV>
__global__ void __launch_bounds__(mtc::THREADS, 1) pa_mass_tc_kernel(MassParams P, int nt, int rows_c, int chunks) {
    using namespace mtc;
    using Y = Lay<D>;
    constexpr int BITS = KV == PA_INT4 ? 4 : (KV == PA_E4M3 || KV == PA_INT8) ? 8 : 16;
    constexpr bool BF = KV == PA_BF16;
    constexpr int NA = Y::NA;
    constexpr int RB = D * BITS / 8, PR = RB / 16;  // bytes and 16-byte pieces per token
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Y::BAR_OFF);
    int *misc = reinterpret_cast<int *>(smem + Y::MISC_OFF);
    volatile int *abort = misc + 1;
    int *ps = reinterpret_cast<int *>(smem + Y::PS_OFF);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float NaN = __int_as_float(0x7fc00000);
    if (sb & 1023) {
        if (tid == 0 && P.dev_error) atomicOr(P.dev_error, PA_DEV_ERR_TIMEOUT);
        return;
    }
    const bool bad_len = scan_units<THREADS, CH>(P, ps, misc + 4);
    if (bad_len && blockIdx.x == 0 && P.dev_error) atomicOr(P.dev_error, PA_DEV_ERR_CONTEXT_LEN);
    const long long N = (long long)ps[P.B] * P.Hkv;
    const long long x0 = blockIdx.x * N / gridDim.x, x1 = (blockIdx.x + 1) * N / gridDim.x;
    if (x0 >= x1) return;

    if (tid == 0) {
        for (int i = 0; i < Y::NBARS; ++i) {
            uint32_t c = 1;
            if ((i >= Y::B_AFULL && i < Y::B_AFULL + NA) || (i >= Y::B_SFREE && i < Y::B_SFREE + 2)) c = 4;
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
    const uint32_t tmem = (uint32_t)misc[0];
    uint32_t err = 0;
    Walk w;
    w.x = x0;
    w.x1 = x1;
    w.end = false;
    walk_piece(w, P, ps);

    if (warp < W_EPI) {
        // ================================================== loaders: tile i by warpgroup i & 1
        const int wg = warp >> 2, wq = warp & 3;  // the warp's 32 tokens: 32 wq ..
        int i = 0;
        auto skip = [&](int k) {
            for (int q = 0; q < k && !w.end; ++q) {
                walk_next(w, P, ps, chunks);
                ++i;
            }
        };
        auto ids_of = [&](const Walk &v, int *id) {  // blocks of the warp's two halves of 16 tokens
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = v.u * CH + 32 * wq + 16 * h;
                id[h] = (!v.end && t < v.L) ? P.block_table[(size_t)v.b * P.tbl + t / P.bs] : 0;
            }
        };
        // global address of piece k (of PR) of this lane, and whether it is a token's
        auto piece = [&](const Walk &v, const int *id, int k, bool &live) -> const uint8_t * {
            const int q = k * 32 + lane, t = 32 * wq + q / PR;
            const int blk = k < PR / 2 ? id[0] : id[1];
            live = !v.end && v.u * CH + t < v.L && blk >= 1 && blk < P.num_blocks;
            return P.k_pool + (size_t)(live ? blk : 0) * P.k_block +
                   ((size_t)v.g * P.bs + (v.u * CH + t) % P.bs) * RB + (q % PR) * 16;
        };
        skip(wg);
        if constexpr (BITS == 16) {
            int id[2], issued = 0, done = 0;
            Walk ahead = w;
            ids_of(ahead, id);
            // keep up to PF tiles of this warpgroup in flight, then publish the oldest
            constexpr int PF = NA > 2 ? 2 : 1;
            int ai = i;
            bool ok = true;
            while (ok && (done < issued || !ahead.end)) {
                if (!ahead.end && issued - done < PF) {
                    const int slot = ai % NA;
                    if (ai >= NA && !warp_wait(&bars[Y::B_AFREE + slot], (ai / NA - 1) & 1, abort, err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sb + Y::A_OFF + slot * Y::A_BYTES;
#pragma unroll 4
                    for (int k = 0; k < PR; ++k) {
                        bool live;
                        const uint8_t *src = piece(ahead, id, k, live);
                        const int q = k * 32 + lane;
                        cp_async16(dst + op_off(CH, 32 * wq + q / PR, q % PR), src, live);
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    ++issued;
                    for (int q = 0; q < 2 && !ahead.end; ++q) walk_next(ahead, P, ps, chunks);
                    ai += 2;
                    ids_of(ahead, id);
                    if (!ahead.end && issued - done < PF) continue;
                }
                if (issued - done > 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
                else asm volatile("cp.async.wait_group 0;" ::: "memory");
                fence_proxy_async_smem();
                warp_arrive(&bars[Y::B_AFULL + (i + 2 * done) % NA]);
                ++done;
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        } else {
            int id[2], id2[2];
            ids_of(w, id);
            uint4 raw[PR];
            auto fetch = [&]() {
#pragma unroll
                for (int k = 0; k < PR; ++k) {
                    bool live;
                    const uint8_t *src = piece(w, id, k, live);
                    raw[k] = live ? __ldg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0u, 0u, 0u, 0u);
                }
            };
            fetch();
            Walk v = w;
            for (int q = 0; q < 2 && !v.end; ++q) walk_next(v, P, ps, chunks);
            ids_of(v, id2);
            while (!w.end) {
                const int slot = i % NA;
                if (i >= NA && !warp_wait(&bars[Y::B_AFREE + slot], (i / NA - 1) & 1, abort, err)) break;
                uint8_t *dst = smem + Y::A_OFF + slot * Y::A_BYTES;
                constexpr int OC = 16 / BITS;  // 16-byte operand chunks per raw piece
#pragma unroll
                for (int k = 0; k < PR; ++k) {
                    uint32_t wd[4 * OC];
                    decode<KV>(raw[k], wd);
                    const int q = k * 32 + lane, t = 32 * wq + q / PR, c = (q % PR) * OC;
#pragma unroll
                    for (int o = 0; o < OC; ++o)
                        *reinterpret_cast<uint4 *>(dst + op_off(CH, t, c + o)) =
                            make_uint4(wd[4 * o], wd[4 * o + 1], wd[4 * o + 2], wd[4 * o + 3]);
                }
                // the next tile of this warpgroup: its blocks are known, load it now
                w = v;
                id[0] = id2[0];
                id[1] = id2[1];
                fetch();
                fence_proxy_async_smem();
                warp_arrive(&bars[Y::B_AFULL + slot]);
                i += 2;
                for (int q = 0; q < 2 && !v.end; ++q) walk_next(v, P, ps, chunks);
                ids_of(v, id2);
            }
        }
    } else if (warp < W_MMA) {
        // ================================================== sums over rows; query staging
        const int wg = (warp - W_EPI) >> 2, qd = warp & 3;
        const int t = 32 * qd + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16) + 256u * wg;
        const int rp = (rows_c + 7) / 8 * 8;                    // rows of a term in the B operand
        int seg = -1, pb = -1, pg = -1, pc = -1, sphase = 0, pua = -1;
        bool ok = true;
        for (; !w.end && ok; walk_next(w, P, ps, chunks)) {
            if (w.b != pb || w.g != pg || w.c != pc || w.ua != pua) {
                // a new segment: its query rows, one warp per row
                ++seg;
                pb = w.b;
                pg = w.g;
                pc = w.c;
                pua = w.ua;
                if (seg > 0 && !warp_wait(&bars[Y::B_QFREE], (seg - 1) & 1, abort, err)) {
                    ok = false;
                    break;
                }
                float *cst = reinterpret_cast<float *>(smem + Y::CST_OFF) + (seg & 1) * (Y::NMAX / 2) * 4;
                int *vs = reinterpret_cast<int *>(smem + Y::VIS_OFF) + (seg & 1) * Y::NMAX;
                const float *fold = P.k_mode == PA_SCALE_CHANNEL ? P.k_scale + (size_t)w.g * D : nullptr;
                const bool scaled = !BF && (fold != nullptr || P.q_dtype == PA_BF16);
                for (int rr = warp - W_EPI; rr < rp; rr += 8) {
                    const int r = w.c * rows_c + rr;
                    const bool rok = rr < rows_c && r < P.R;
                    const int j = rok ? r / P.G : 0, h = w.g * P.G + (rok ? r % P.G : 0);
                    const size_t row = ((size_t)w.b * P.n + j) * P.Hq + h;
                    const uint8_t *src = P.q + row * (2 * D);
                    // lane: operand words lane, lane + 32, ... (pairs of channels)
                    float v[D / 64][2], mx = 0.f;
#pragma unroll
                    for (int i = 0; i < D / 64; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int word = lane + 32 * i;
                            constexpr int WP = 64 / BITS;  // words per raw piece
                            const int ch = channel_of<BITS>(word / WP, word % WP, e);
                            v[i][e] = rok ? q_val(src, ch, P.q_dtype) * (fold ? fold[ch] : 1.f) : 0.f;
                            mx = fmaxf(mx, fabsf(v[i][e]));
                        }
                    float down = 1.f;
                    if (scaled) {
#pragma unroll
                        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        int ex = 0;
                        if (mx > 0.f && mx < 3.0e38f) frexpf(mx, &ex);
                        ex = max(-120, min(120, ex));
                        const float up = __int_as_float((127 - ex) << 23);
                        down = __int_as_float((127 + ex) << 23);
#pragma unroll
                        for (int i = 0; i < D / 64; ++i) {
                            v[i][0] *= up;
                            v[i][1] *= up;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) {
                        const int word = lane + 32 * i, c = word >> 2;
                        float a = v[i][0], d = v[i][1];
                        for (int q = 0; q < nt; ++q) {
                            const uint32_t x = pack2<BF>(a, d);
                            *reinterpret_cast<uint32_t *>(smem + Y::Q_OFF + op_off(nt * rp, q * rp + rr, c) +
                                                          4 * (word & 3)) = x;
                            if constexpr (BF) {
                                a -= __uint_as_float(x << 16);
                                d -= __uint_as_float(x & 0xFFFF0000u);
                            } else {
                                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
                                a -= f.x;
                                d -= f.y;
                            }
                        }
                    }
                    if (lane == 0) {
                        const float ks = P.k_mode == PA_SCALE_TENSOR ? P.k_scale[0] : 1.f;
                        const float lse = rok ? P.lse[row] : -INFINITY;
                        const bool on = rok && lse != -INFINITY;
                        cst[(rr >> 1) * 4 + (rr & 1)] = on ? P.softmax_scale * ks * down : 0.f;
                        cst[(rr >> 1) * 4 + 2 + (rr & 1)] = on ? -lse : -INFINITY;
                        // rows past R never count, and do not force the masked sum either
                        vs[rr] = !rok ? 0x7FFFFFFF : !on ? 0 : P.causal ? w.L - (P.n - 1 - j) : w.L;
                    }
                }
                fence_proxy_async_smem();
                warp_arrive(&bars[Y::B_QFULL]);
                if (!warp_wait(&bars[Y::B_QFULL], seg & 1, abort, err)) {
                    ok = false;
                    break;
                }
            }
            if ((w.u & 1) != wg) continue;
            const int tok = w.u * CH + t;
            const bool in = tok < w.L;
            const int blk = in ? P.block_table[(size_t)w.b * P.tbl + tok / P.bs] : 0;
            const bool okb = blk >= 1 && blk < P.num_blocks;
            float ts = 1.f;
            if (KV == PA_E4M3 && P.k_mode == PA_SCALE_TOKEN && in && okb)
                ts = __ldg(reinterpret_cast<const float *>(P.k_pool + (size_t)blk * P.k_block + P.k_codes) +
                           (size_t)w.g * P.bs + tok % P.bs);
            float *out = P.mass + ((size_t)w.b * P.Hkv + w.g) * P.max_ctx + tok;
            const float dec = w.c == 0 ? P.decay : 1.f;
            const float old = in && dec != 0.f ? *out : 0.f;
            const float4 *cst = reinterpret_cast<const float4 *>(smem + Y::CST_OFF) + (seg & 1) * (Y::NMAX / 2);
            const int *vs = reinterpret_cast<const int *>(smem + Y::VIS_OFF) + (seg & 1) * Y::NMAX;
            bool masked = false;
            if (w.u * CH + CH > w.L - P.n) {
                masked = true;
            } else {  // a row that saw nothing (lse = -inf) is masked everywhere
                int mn = 0x7FFFFFFF;
                for (int r = lane; r < rp; r += 32) mn = min(mn, vs[r]);
                masked = __any_sync(0xffffffffu, mn <= 0);
            }
            ok = warp_wait_u(&bars[Y::B_SFULL + wg], sphase & 1, abort, err);
            if (!ok) break;
            ++sphase;
            tc_fence_after();
            float tot[4] = {0.f, 0.f, 0.f, 0.f};
            for (int r0 = 0; r0 < rp; r0 += 8) {
                uint32_t z[8], z2[8];
                tmem_ld8_nowait(tl + (uint32_t)r0, z);
                if (nt == 2) tmem_ld8_nowait(tl + (uint32_t)(rp + r0), z2);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 c4 = cst[(r0 + e) >> 1];
                    float a = __uint_as_float(z[e]), d = __uint_as_float(z[e + 1]);
                    if (nt == 2) {
                        a += __uint_as_float(z2[e]);
                        d += __uint_as_float(z2[e + 1]);
                    }
                    const float pa_ = ex2(fmaf(a * ts, c4.x, c4.z) * LOG2E);
                    const float pd = ex2(fmaf(d * ts, c4.y, c4.w) * LOG2E);
                    if (masked) {
                        const int2 v2 = *reinterpret_cast<const int2 *>(vs + r0 + e);
                        tot[e & 2] += tok < v2.x ? pa_ : 0.f;
                        tot[(e & 2) + 1] += tok < v2.y ? pd : 0.f;
                    } else {
                        tot[e & 2] += pa_;
                        tot[(e & 2) + 1] += pd;
                    }
                }
            }
            tc_fence_before();
            warp_arrive(&bars[Y::B_SFREE + wg]);
            if (in) {
                const float got = (tot[0] + tot[1]) + (tot[2] + tot[3]);
                *out = !okb ? NaN : dec != 0.f ? fmaf(dec, old, got) : got;
                if (!okb) err |= PA_DEV_ERR_BLOCK_ID;
            }
        }
        if (!ok) {  // a wait ran out: the rest of the share is NaN
            for (; !w.end; walk_next(w, P, ps, chunks)) {
                const int tok = w.u * CH + t;
                if ((w.u & 1) == wg && tok < w.L) P.mass[((size_t)w.b * P.Hkv + w.g) * P.max_ctx + tok] = NaN;
            }
        }
    } else {
        // ================================================== MMA issue (lane 0)
        if (lane == 0) {
            const int rp = (rows_c + 7) / 8 * 8, n = nt * rp;
            constexpr uint32_t FMT = BF ? (1u << 7) | (1u << 10) : 0u;
            const uint32_t id = idesc(CH, (n + 15) / 16 * 16, 0) | FMT;
            int i = 0, seg = -1, pb = -1, pg = -1, pc = -1, pua = -1;
            int used[2] = {0, 0};
            for (; !w.end; ++i) {
                if (w.b != pb || w.g != pg || w.c != pc || w.ua != pua) {
                    ++seg;
                    pb = w.b;
                    pg = w.g;
                    pc = w.c;
                    pua = w.ua;
                    if (!lane_wait(&bars[Y::B_QFULL], seg & 1, abort, err)) break;
                }
                const int slot = i % NA, buf = w.u & 1;
                if (!lane_wait(&bars[Y::B_AFULL + slot], (i / NA) & 1, abort, err)) break;
                if (used[buf] > 0 && !lane_wait(&bars[Y::B_SFREE + buf], (used[buf] - 1) & 1, abort, err)) break;
                ++used[buf];
                tc_fence_after();
                const uint64_t a = sdesc(sb + Y::A_OFF + slot * Y::A_BYTES, 16, 1024, 2);
                const uint64_t q = sdesc(sb + Y::Q_OFF, 16, 1024, 2);
                for (int k = 0; k < D / 16; ++k)
                    mma_f16(tmem + 256u * buf, a + (uint32_t)(((k >> 2) * CH * 128 + 32 * (k & 3)) >> 4),
                            q + (uint32_t)(((k >> 2) * n * 128 + 32 * (k & 3)) >> 4), id, k > 0 ? 1u : 0u);
                mma_commit(&bars[Y::B_SFULL + buf]);
                mma_commit(&bars[Y::B_AFREE + slot]);
                walk_next(w, P, ps, chunks);
                if (w.end || w.b != pb || w.g != pg || w.c != pc || w.ua != pua) mma_commit(&bars[Y::B_QFREE]);
            }
            mma_commit(&bars[Y::B_DONE]);
            (void)mbar_wait_bounded(&bars[Y::B_DONE], 0, nullptr);
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
    const int smem = Y::PS_OFF + (P.B + 1) * 4;
    if (smem > 227 * 1024) return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev >= 64 || !(done.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(pa_mass_tc_kernel<D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    // chunks of rows of equal size, as few as fit the operand
    const int most = Y::NMAX / nt, chunks = (P.R + most - 1) / most;
    int rows_c = (P.R + chunks - 1) / chunks;
    rows_c = (rows_c + 15) / 16 * 16;  // (a multiple of the MMA's N step, also with two terms side by side)
    // no CTA without a tile of the longest possible batch
    const long long tiles = (long long)P.B * P.Hkv * ((P.max_ctx + mtc::CH - 1) / mtc::CH);
    const int ctas = (int)std::max(1ll, std::min<long long>(sms, tiles));
    pa_mass_tc_kernel<D, KV><<<ctas, mtc::THREADS, smem, s>>>(P, nt, rows_c, (P.R + rows_c - 1) / rows_c);
    return cudaPeekAtLastError();
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
