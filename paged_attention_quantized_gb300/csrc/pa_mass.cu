// Accumulated attention weight of the cached tokens:
//
//   mass[b][g][t] = decay mass[b][g][t]
//                   + sum over query rows r of kv head g that see t of exp(c q_r . k_t - lse_r)
//
// The log-sum-exp is an input, so one pass over K suffices: a token's sum is
// over rows, not over tokens, and no state is carried between tokens.  HBM
// bound at decode: every K row is read once.  Measured on a GB300: one row of
// 32 / 8 heads over 64 requests of 512-8192 tokens, bf16 head dim 128, 108 us =
// 6.0 TB/s (0.89 of the measured copy rate); four tokens (16 rows per
// kv head) of 32 requests of 1024-32768, E4M3 head dim 256, 285 us = 4.5 TB/s (0.67: some 400
// instructions per 16 tokens, half of them conversions).
//
// Tokens are the M axis of mma.sync (S^T = K q^T): a warp holds 16 tokens of
// one (request, kv head), the query rows are N, and a token's sum is a sum
// over the accumulator's columns -- in registers, then across the four lanes
// that share a token.  K goes straight from global memory into the operand
// registers: lane i of a quad reads 16-byte pieces i, i + 4, ... of its two
// rows, and the channel order this gives the contraction is applied to q as
// well.  Units of 16 tokens in logical order (request, kv head, unit) are
// shared evenly by persistent warps; each knows its share from a prefix sum
// over context_lens that every CTA computes for itself.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "pa_mass.cuh"

namespace pa {
namespace mass {

constexpr int THREADS = 256, UT = 16;  // tokens per unit

// What a warp needs to know of a unit; its block id is asked for a unit before
// its rows, its rows a unit before they are used.
struct Unit {
    int b, g, u, L, units, blk;  // (b = P.B: none)
};

// NB blocks of 8 query rows; NT terms per query value.  Query operands stay in
// registers while they take at most 32 of them a lane; beyond (16 rows of head
// dim 256, say) each warp keeps its own in shared memory, in the order its lanes
// use them, so that twice as many warps are resident.  PF: whether the next
// unit's rows are loaded while this one is used (row pieces of both must fit the
// registers).  Measured, 4.4 M tokens of 8 kv heads: 16 rows of E4M3 head dim 256
// 4.56 TB/s (4.37 with the operands in registers and no rows ahead), bf16 head
// dim 128 with 4 rows 5.95 TB/s (5.98).
template <int D, int KV, int NB, int NT>
struct Shape {
    static constexpr int BITS = KV == PA_INT4 ? 4 : (KV == PA_E4M3 || KV == PA_INT8) ? 8 : 16;
    static constexpr int PIECES = D * BITS / 8 / 64;  // 16-byte pieces per lane and row
    static constexpr int WORDS = 64 / BITS;           // operand words per piece
    static constexpr int QW = PIECES * WORDS;         // operand words per lane and query row
    static constexpr bool QS = NB * NT * QW > 32;
    static constexpr bool PF = PIECES <= 4;
    static constexpr int Q_BYTES = QS ? NB * NT * QW * 128 : 0;  // per warp
    static constexpr int CTAS = D == 64 && NB * NT == 1 ? 3 : 2;   // resident CTAs the registers are held to
};

template <int D, int KV, int NB, int NT>
__global__ void __launch_bounds__(THREADS, Shape<D, KV, NB, NT>::CTAS) pa_mass_kernel(MassParams P) {
    using S = Shape<D, KV, NB, NT>;
    constexpr int BITS = S::BITS, PIECES = S::PIECES, WORDS = S::WORDS, QW = S::QW;
    constexpr bool BF = KV == PA_BF16, QS = S::QS;
    extern __shared__ __align__(16) uint8_t smem[];
    int *ps = reinterpret_cast<int *>(smem + THREADS / 32 * S::Q_BYTES);  // units before request b (B + 1 entries)
    __shared__ int warp_tot[THREADS / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float NaN = __int_as_float(0x7fc00000);

    grid_dependents_launch();
    grid_dependency_wait();
    const bool bad_len = scan_units<THREADS, UT>(P, ps, warp_tot);
    if (bad_len && blockIdx.x == 0 && P.dev_error) atomicOr(P.dev_error, PA_DEV_ERR_CONTEXT_LEN);
    const long long N = (long long)ps[P.B] * P.Hkv;
    const long long W = (long long)gridDim.x * (THREADS / 32), k = (long long)blockIdx.x * (THREADS / 32) + warp;
    const long long x0 = k * N / W, x1 = (k + 1) * N / W;
    if (x0 >= x1) return;

    const int gr = lane >> 2, qi = lane & 3;
    uint32_t qr[QS ? 1 : NB * NT * QW];
    uint32_t *qs = reinterpret_cast<uint32_t *>(smem + warp * S::Q_BYTES) + lane * 4;  // [4 words][32 lanes][4]
    float sc[NB][2], ls[NB][2];
    int vis[NB][2];

    // operand words of the query rows of (b, g), and the constants of the rows whose
    // columns this lane's accumulators hold (2 qi, 2 qi + 1)
    auto load_q = [&](int b, int g, int L) {
        if (QS) __syncwarp();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int r = nb * 8 + gr;
            const bool ok = r < P.R;
            const int j = ok ? r / P.G : 0, h = g * P.G + (ok ? r % P.G : 0);
            const size_t row = ((size_t)b * P.n + j) * P.Hq + h;
            const uint8_t *src = P.q + row * (2 * D);
            const float *fold = P.k_mode == PA_SCALE_CHANNEL ? P.k_scale + (size_t)g * D : nullptr;
            // f16 operands of other queries than plain f16 ones are scaled by a power of two into [-1, 1)
            const bool scaled = !BF && (fold != nullptr || P.q_dtype == PA_BF16);
            float mx = 0.f;
            if (scaled) {
#pragma unroll 4
                for (int i = 0; i < QW; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int ch = channel_of<BITS>((i / WORDS) * 4 + qi, i % WORDS, e);
                        const float v = ok ? q_val(src, ch, P.q_dtype) * (fold ? fold[ch] : 1.f) : 0.f;
                        mx = fmaxf(mx, fabsf(v));
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            }
            int ex = 0;
            if (mx > 0.f && mx < 3.0e38f) frexpf(mx, &ex);
            ex = max(-120, min(120, ex));
            const float up = __int_as_float((127 - ex) << 23), down = __int_as_float((127 + ex) << 23);
#pragma unroll
            for (int i = 0; i < QW; ++i) {
                float v[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int ch = channel_of<BITS>((i / WORDS) * 4 + qi, i % WORDS, e);
                    v[e] = ok ? q_val(src, ch, P.q_dtype) * (fold ? fold[ch] : 1.f) : 0.f;
                    if (scaled) v[e] *= up;
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint32_t x = pack2<BF>(v[0], v[1]);
                    const int at = (nb * NT + t) * QW + i;
                    if constexpr (QS) qs[(at >> 2) * 128 + (at & 3)] = x;
                    else qr[at] = x;
                    if (t + 1 < NT) {
                        if constexpr (BF) {
                            v[0] -= __uint_as_float(x << 16);
                            v[1] -= __uint_as_float(x & 0xFFFF0000u);
                        } else {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
                            v[0] -= f.x;
                            v[1] -= f.y;
                        }
                    }
                }
            }
            const float ks = P.k_mode == PA_SCALE_TENSOR ? P.k_scale[0] : 1.f;
            const float mysc = P.softmax_scale * ks * down;
            const float myls = ok ? P.lse[row] : 0.f;
            const int myvis = (!ok || myls == -INFINITY) ? 0 : P.causal ? L - (P.n - 1 - j) : L;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int from = (2 * qi + e) * 4;
                sc[nb][e] = __shfl_sync(0xffffffffu, mysc, from);
                ls[nb][e] = __shfl_sync(0xffffffffu, myls, from);
                vis[nb][e] = __shfl_sync(0xffffffffu, myvis, from);
            }
        }
        if (QS) __syncwarp();
    };

    long long left = x1 - x0;  // units from cur on
    auto with_block = [&](Unit &n) {
        const int t0 = n.u * UT;
        n.blk = n.b < P.B ? P.block_table[(size_t)n.b * P.tbl + __umulhi((unsigned)t0, P.bs_mul)] : 0;
    };
    auto after = [&](const Unit &c, bool any) -> Unit {  // the next unit in logical order, its block asked for
        Unit n = c;
        if (!any) n.b = P.B;
        if (n.b < P.B && ++n.u == n.units) {
            n.u = 0;
            if (++n.g == P.Hkv) {
                n.g = 0;
                do ++n.b;
                while (n.b < P.B && ps[n.b + 1] == ps[n.b]);
                if (n.b < P.B) {
                    n.units = ps[n.b + 1] - ps[n.b];
                    n.L = P.context_lens[n.b];
                }
            }
        }
        with_block(n);
        return n;
    };
    struct Rows {
        uint4 raw[2][PIECES];
        float ts[2], old;
    };
    auto load = [&](const Unit &c, Rows &r) {
        if (c.b >= P.B) return;
        const bool okb = c.blk >= 1 && c.blk < P.num_blocks;
        const int t0 = c.u * UT, slot = t0 - (int)__umulhi((unsigned)t0, P.bs_mul) * P.bs;
        const uint8_t *base = P.k_pool + (size_t)(okb ? c.blk : 0) * P.k_block;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = c.g * P.bs + slot + gr + 8 * e;
            const uint4 *src = reinterpret_cast<const uint4 *>(base + (size_t)row * (D * BITS / 8));
            const bool live = okb && t0 + gr + 8 * e < c.L;
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
                r.raw[e][i] = live ? __ldg(src + 4 * i + qi) : make_uint4(0u, 0u, 0u, 0u);
            r.ts[e] = 1.f;
            if (KV == PA_E4M3 && P.k_mode == PA_SCALE_TOKEN && live)
                r.ts[e] = __ldg(reinterpret_cast<const float *>(base + P.k_codes) + row);
        }
        // lane 0 of a quad writes token gr, lane 1 token gr + 8
        const int tok = t0 + gr + 8 * qi;
        r.old = qi < 2 && tok < c.L && P.decay != 0.f ? P.mass[((size_t)c.b * P.Hkv + c.g) * P.max_ctx + tok] : 0.f;
    };
    uint32_t err = 0;
    int qb = -1, qg = -1;
    auto use = [&](const Unit &c, const Rows &r) {
        if (c.b != qb || c.g != qg) {
            load_q(c.b, c.g, c.L);
            qb = c.b;
            qg = c.g;
        }
        const int t0 = c.u * UT, tok[2] = {t0 + gr, t0 + gr + 8};
        float tot[2] = {0.f, 0.f};
        float acc[NB][NT][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nb][t][e] = 0.f;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            uint32_t w0[WORDS], w1[WORDS];
            decode<KV>(r.raw[0][i], w0);
            decode<KV>(r.raw[1][i], w1);
#pragma unroll
            for (int s = 0; s < WORDS / 2; s += 2) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const int at = (nb * NT + t) * QW + i * WORDS + 2 * s;  // four words: two steps
                        uint32_t q[4];
                        if constexpr (QS) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(qs + (at >> 2) * 128);
                            q[0] = v.x;
                            q[1] = v.y;
                            q[2] = v.z;
                            q[3] = v.w;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) q[e] = qr[at + e];
                        }
                        const uint32_t a0[4] = {w0[2 * s], w1[2 * s], w0[2 * s + 1], w1[2 * s + 1]};
                        const uint32_t a1[4] = {w0[2 * s + 2], w1[2 * s + 2], w0[2 * s + 3], w1[2 * s + 3]};
                        mma16816<BF>(acc[nb][t], a0, q[0], q[1]);
                        mma16816<BF>(acc[nb][t], a1, q[2], q[3]);
                    }
            }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float z = NT == 2 ? acc[nb][0][e] + acc[nb][NT - 1][e] : acc[nb][0][e];
                const float d = fmaf(z * r.ts[e >> 1], sc[nb][e & 1], -ls[nb][e & 1]);
                const float p = ex2(d * LOG2E);
                tot[e >> 1] += tok[e >> 1] < vis[nb][e & 1] ? p : 0.f;
            }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            tot[e] += __shfl_xor_sync(0xffffffffu, tot[e], 1);
            tot[e] += __shfl_xor_sync(0xffffffffu, tot[e], 2);
        }
        const bool okb = c.blk >= 1 && c.blk < P.num_blocks;
        if (!okb) err |= PA_DEV_ERR_BLOCK_ID;
        const int mytok = t0 + gr + 8 * qi;
        if (qi < 2 && mytok < c.L) {
            const float got = qi == 0 ? tot[0] : tot[1];
            P.mass[((size_t)c.b * P.Hkv + c.g) * P.max_ctx + mytok] =
                !okb ? NaN : P.decay != 0.f ? fmaf(P.decay, r.old, got) : got;
        }
    };

    Unit cur;
    cur.b = request_of(ps, P.B, (int)(x0 / P.Hkv));
    {
        const long long rem = x0 - (long long)ps[cur.b] * P.Hkv;
        cur.units = ps[cur.b + 1] - ps[cur.b];
        cur.g = (int)(rem / cur.units);
        cur.u = (int)(rem % cur.units);
        cur.L = P.context_lens[cur.b];
        with_block(cur);
    }
    Unit nxt = after(cur, left > 1);
    if constexpr (S::PF) {
        Rows r0, r1;
        load(cur, r0);
        while (true) {
            Unit nn = after(nxt, left > 2);
            load(nxt, r1);
            use(cur, r0);
            if (--left == 0) break;
            cur = nxt;
            nxt = nn;
            nn = after(nxt, left > 2);
            load(nxt, r0);
            use(cur, r1);
            if (--left == 0) break;
            cur = nxt;
            nxt = nn;
        }
    } else {
        Rows r;
        while (true) {
            const Unit nn = after(nxt, left > 2);
            load(cur, r);
            use(cur, r);
            if (--left == 0) break;
            cur = nxt;
            nxt = nn;
        }
    }
    if (err && lane == 0 && P.dev_error) atomicOr(P.dev_error, err);
}

template <int D, int KV, int NB, int NT>
cudaError_t launch_rows(const MassParams &P, int sms, cudaStream_t s) {
    using S = Shape<D, KV, NB, NT>;
    constexpr int QB = THREADS / 32 * S::Q_BYTES;
    const int smem = QB + (P.B + 1) * 4;
    // resident CTAs, asked for once per device at the largest prefix-sum array that
    // leaves them all room (more requests: asked again)
    static std::atomic<int> kept[64];
    int dev = 0, per = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev < 64 && P.B < 1024;
    if (keep) per = kept[dev].load(std::memory_order_relaxed);
    if (per == 0) {
        if (QB + (MAX_B + 1) * 4 > 48 * 1024) {
            e = cudaFuncSetAttribute(pa_mass_kernel<D, KV, NB, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     QB + (MAX_B + 1) * 4);
            if (e != cudaSuccess) return e;
        }
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, pa_mass_kernel<D, KV, NB, NT>, THREADS,
                                                          keep ? QB + 4096 : smem);
        if (e != cudaSuccess) return e;
        per = std::max(1, per);
        if (keep) kept[dev].store(per, std::memory_order_relaxed);
    }
    // no warp without a unit of the longest possible batch
    const long long units = (long long)P.B * P.Hkv * ((P.max_ctx + UT - 1) / UT);
    const long long ctas = std::min<long long>((long long)sms * per, (units + THREADS / 32 - 1) / (THREADS / 32));
    return launch_pdl(pa_mass_kernel<D, KV, NB, NT>, dim3((unsigned)ctas), dim3(THREADS), (size_t)smem, s, P);
}

template <int D, int KV, int NT>
cudaError_t launch(const MassParams &P, int sms, cudaStream_t s) {
    // (more rows of 16-bit codes of head dims 128 and 256 go to the tensor-core kernel)
    if constexpr (D == 64 || (KV != PA_F16 && KV != PA_BF16))
        if (P.R > 8) return launch_rows<D, KV, 2, NT>(P, sms, s);
    return launch_rows<D, KV, 1, NT>(P, sms, s);
}

// query terms: a folded per-channel scale, and f16 queries (11 bits) against
// bf16 operands, need two
int query_terms(const MassParams &P, int kv) {
    return (P.k_mode == PA_SCALE_CHANNEL || (kv == PA_BF16 && P.q_dtype == PA_F16)) ? 2 : 1;
}

template <int D>
cudaError_t dispatch(const MassParams &P, int kv, int sms, cudaStream_t s) {
    const bool two = query_terms(P, kv) == 2;
    switch (kv) {
        case PA_F16: return launch<D, PA_F16, 1>(P, sms, s);
        case PA_BF16: return two ? launch<D, PA_BF16, 2>(P, sms, s) : launch<D, PA_BF16, 1>(P, sms, s);
        case PA_E4M3: return two ? launch<D, PA_E4M3, 2>(P, sms, s) : launch<D, PA_E4M3, 1>(P, sms, s);
        case PA_INT8: return two ? launch<D, PA_INT8, 2>(P, sms, s) : launch<D, PA_INT8, 1>(P, sms, s);
        case PA_INT4:
            if constexpr (D >= 128) return two ? launch<D, PA_INT4, 2>(P, sms, s) : launch<D, PA_INT4, 1>(P, sms, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace mass
}  // namespace pa

extern "C" PA_API pa_status pa_attention_mass(const pa_problem *p, float decay, const void *q, const void *k_pool,
                                              const int32_t *block_table, const int32_t *context_lens,
                                              const float *k_scale, const float *lse, float *mass, uint32_t *dev_error,
                                              pa_stream_t stream) {
    if (p == nullptr) return PA_ERR_INVALID_ARG;
    if (p->batch < 0 || p->next_n < 1 || p->num_q_heads < 1 || p->num_kv_heads < 1 ||
        p->num_q_heads % p->num_kv_heads != 0 || p->head_dim_k < 1 || p->block_size < 1 || p->num_blocks < 1 ||
        p->max_blocks_per_seq < 1 || p->max_context_len < 0 || p->num_sms < 0)
        return PA_ERR_INVALID_ARG;
    if ((p->q_dtype != PA_F16 && p->q_dtype != PA_BF16) || p->kv_dtype < PA_F16 || p->kv_dtype > PA_INT4 ||
        p->k_scale_mode < PA_SCALE_NONE || p->k_scale_mode > PA_SCALE_TOKEN || (p->causal != 0 && p->causal != 1) ||
        !std::isfinite(p->softmax_scale) || !std::isfinite(decay))
        return PA_ERR_INVALID_ARG;
    const int D = p->head_dim_k, kv = p->kv_dtype;
    if ((D != 64 && D != 128 && D != 256) || (kv == PA_INT4 && D == 64) || p->block_size % 16 != 0 ||
        p->batch > pa::mass::MAX_B)
        return PA_ERR_UNSUPPORTED;
    const bool half = kv == PA_F16 || kv == PA_BF16;
    if ((half && p->k_scale_mode > PA_SCALE_TENSOR) || (kv != PA_E4M3 && p->k_scale_mode == PA_SCALE_TOKEN))
        return PA_ERR_UNSUPPORTED;
    const int G = p->num_q_heads / p->num_kv_heads;
    const long long R = (long long)G * p->next_n;
    const int bits = half ? 16 : kv == PA_INT4 ? 4 : 8;
    const long long codes = (long long)p->num_kv_heads * p->block_size * (D * bits / 8);
    // units of 16 tokens are counted in 32 bits, over the batch
    if (R > (1 << 20) || codes > 0x7FFFFFFFll ||
        ((long long)p->max_context_len + 128) * p->block_size >= (1ll << 32) ||
        (long long)p->batch * (p->max_context_len / 16 + 1) > 0x7FFFFFFFll)
        return PA_ERR_UNSUPPORTED;
    if (p->batch == 0 || p->max_context_len == 0) return PA_OK;
    if (q == nullptr || k_pool == nullptr || block_table == nullptr || context_lens == nullptr || lse == nullptr ||
        mass == nullptr ||
        ((p->k_scale_mode == PA_SCALE_TENSOR || p->k_scale_mode == PA_SCALE_CHANNEL) && k_scale == nullptr))
        return PA_ERR_INVALID_ARG;
    auto off = [](const void *x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) & (a - 1)) != 0; };
    if (off(q, 16) || off(k_pool, 16) || off(block_table, 4) || off(context_lens, 4) || off(lse, 4) || off(mass, 4) ||
        off(k_scale, 4) || off(dev_error, 4))
        return PA_ERR_INVALID_ARG;
    int sms = p->num_sms;
    if (sms == 0) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return PA_ERR_CUDA;
    }
    pa::MassParams P;
    P.q = static_cast<const uint8_t *>(q);
    P.k_pool = static_cast<const uint8_t *>(k_pool);
    P.block_table = block_table;
    P.context_lens = context_lens;
    P.k_scale = k_scale;
    P.lse = lse;
    P.mass = mass;
    P.dev_error = dev_error;
    P.k_block = codes + (p->k_scale_mode == PA_SCALE_TOKEN ? (long long)p->num_kv_heads * p->block_size * 4 : 0);
    P.k_codes = (int)codes;
    P.B = p->batch;
    P.n = p->next_n;
    P.Hq = p->num_q_heads;
    P.Hkv = p->num_kv_heads;
    P.G = G;
    P.R = (int)R;
    P.bs = p->block_size;
    P.tbl = p->max_blocks_per_seq;
    P.max_ctx = p->max_context_len;
    P.num_blocks = p->num_blocks;
    P.q_dtype = p->q_dtype;
    P.k_mode = p->k_scale_mode;
    P.causal = p->causal;
    P.bs_mul = (unsigned)((1ull << 32) / (unsigned)p->block_size) + 1u;
    P.decay = decay;
    P.softmax_scale = p->softmax_scale;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // Past 16 rows the tensor-core kernel; up to 8, and at head dim 64, this one.
    // Between (16 rows, 8 kv heads, this one / the other): 16-bit codes of head dim
    // 128 over 64 requests of 512-8192 tokens 156 / 125 us.  Quantized codes cost the
    // other one its change from (request, kv head) to the next, so it takes them while
    // they are few: two requests of 37-70 tokens, E4M3 head dim 256, 19.6 / 6.2 us, one
    // of 20000-32768 39.6 / 23.1, 16 of 2048-16384 118 / 90; 32 of 1024-32768, for two
    // draws of their lengths, 183 / 182 and 285 / 299; 64 of 512-8192, head dim 128, 84 / 109.
    const bool few = (long long)P.B * P.Hkv <= sms;
    const bool tc = P.R > 16 || (P.R > 8 && D > 64 && (kv == PA_F16 || kv == PA_BF16 || few));
    const cudaError_t e = tc         ? pa::mass::launch_mass_tc(P, kv, D, pa::mass::query_terms(P, kv), sms, s)
                          : D == 64  ? pa::mass::dispatch<64>(P, kv, sms, s)
                          : D == 128 ? pa::mass::dispatch<128>(P, kv, sms, s)
                                     : pa::mass::dispatch<256>(P, kv, sms, s);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
