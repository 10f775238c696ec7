// Eviction from the paged cache by accumulated attention weight.
//
// Selection (pa_evict_select_kernel), one CTA per (request, kv head): every
// slot gets a 32-bit key that orders as its mass does (protected slots the
// largest key, NaN the smallest), the left-th largest key is found bit by bit
// by counting keys at or above a candidate, and the slots above it plus the
// first of those equal to it are kept.  Keys stay in registers (up to 32
// slots per lane; longer rows read the mass again from L2 for every count).
// Ordered ranks of the free slots below `left` and of the kept ones at or past
// it come from warp ballots and one scan over the warps; their i-th entries
// pair up as the moves of the row.
//
// Moves (pa_evict_move_kernel): one thread per 16-byte piece of a moved K or V
// row.  Sources lie at or past `left`, destinations below it, so no row is
// read after it was written, whatever the order; HBM bound.
#include <algorithm>
#include <cmath>

#include "pa_common.cuh"

namespace pa {

struct EvictParams {
    const float *mass;
    const int32_t *positions;
    const int32_t *history;
    const int32_t *block_table;
    const int32_t *context_lens;
    uint8_t *k_pool;
    uint8_t *v_pool;
    float *mass_out;
    int32_t *positions_out;
    int32_t *history_out;
    int32_t *lens_out;
    uint32_t *hdr;       // workspace: [0] error word
    int4 *req;           // [B] {left, moves allowed (1) or not (0), positions dropped so far, error bits}
    int32_t *counts;     // [B][Hkv] moved rows
    int32_t *lists;      // [B][Hkv][2][cap] destinations, sources
    long long k_block, v_block;  // bytes per pool block
    long long k_codes, v_codes;  // bytes of codes in a block (per-token scales follow)
    int k_row, v_row;            // bytes per row (v_row = 0: no V plane)
    int k_tok, v_tok;            // 1: per-token scales
    int B, Hkv, bs, tbl, max_ctx, num_blocks, budget, sinks, recent, cap;
};

namespace evict {

constexpr int THREADS = 1024, NW = THREADS / 32;
constexpr int MOVE_THREADS = 256, MOVE_ROWS = 32;  // rows of one CTA of the move kernel

// order-preserving key of a mass: larger mass, larger key; NaN below all (0)
__device__ __forceinline__ uint32_t mass_key(float v) {
    if (v != v) return 0u;
    const uint32_t u = __float_as_uint(v + 0.f);  // -0 counts as +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// KPT: slots per lane kept in registers (KPT * 1024 slots), 0 = read again each time
template <int KPT>
__global__ void __launch_bounds__(THREADS) pa_evict_select_kernel(EvictParams P) {
    grid_dependents_launch();  // the move kernel may queue up behind
    __shared__ int s_cnt[32];
    __shared__ int s_warp[3][NW];
    __shared__ uint32_t s_err;
    const int g = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < 32) s_cnt[tid] = 0;
    if (tid == 0) s_err = 0;
    __syncthreads();
    const int L = P.context_lens[b];
    const int base = P.history[2 * b], dropped = P.history[2 * b + 1];
    uint32_t err = 0;
    if (L < 0 || L > P.max_ctx || (long long)L > (long long)P.tbl * P.bs || base < 0 || base > L || dropped < 0 ||
        dropped > 0x7FFFFFFF - L)
        err = PA_DEV_ERR_CONTEXT_LEN;
    if (err == 0) {
        const int pages = (L + P.bs - 1) / P.bs;
        bool badid = false;
        for (int i = tid; i < pages; i += THREADS) {
            const int blk = P.block_table[(size_t)b * P.tbl + i];
            badid |= blk < 1 || blk >= P.num_blocks;
        }
        if (badid) s_err = PA_DEV_ERR_BLOCK_ID;
        __syncthreads();
        err = s_err;
    }
    const int left = min(L, P.budget);
    if (g == 0 && tid == 0) P.req[b] = err ? make_int4(L, base, dropped, (int)err) : make_int4(left, left, dropped + L - left, 0);
    const size_t rowi = (size_t)b * P.Hkv + g;
    if (err) {
        if (tid == 0) P.counts[rowi] = 0;
        return;
    }
    const float *mass = P.mass + rowi * P.max_ctx;
    const int32_t *pos_in = P.positions + rowi * P.max_ctx;
    float *mass_out = P.mass_out + rowi * P.max_ctx;
    int32_t *pos_out = P.positions_out + rowi * P.max_ctx;
    const int newest = L + dropped - P.recent;
    auto pos_of = [&](int s) -> int { return s < base ? pos_in[s] : dropped + s; };
    auto key_of = [&](int s) -> uint32_t {
        const int p = pos_of(s);
        return (p < P.sinks || p >= newest) ? 0xFFFFFFFFu : mass_key(mass[s]);
    };
    // warp w holds slots [w * per, (w + 1) * per), 32 consecutive ones at a time
    const int strips = (L + THREADS - 1) / THREADS;  // strips of 32 per warp
    const int per = strips * 32, s0 = warp * per + lane;
    constexpr int KR = KPT > 0 ? KPT : 1;
    uint32_t key[KR];
    if (KPT > 0) {
#pragma unroll
        for (int i = 0; i < KR; ++i) {
            const int s = s0 + 32 * i;
            key[i] = (i < strips && s < L) ? key_of(s) : 0u;
        }
    }
    // ---- the left-th largest key T: the largest T with at least `left` keys >= T
    uint32_t T = 0;
    int above = L;  // keys >= T
    if (left < L) {
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t cand = T | (1u << bit);
            int n = 0;
            if (KPT > 0) {
#pragma unroll
                for (int i = 0; i < KR; ++i) n += key[i] >= cand ? 1 : 0;  // (unused slots have key 0 < cand)
            } else {
                for (int i = 0; i < strips; ++i) {
                    const int s = s0 + 32 * i;
                    n += (s < L && key_of(s) >= cand) ? 1 : 0;
                }
            }
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0 && n) atomicAdd(&s_cnt[bit], n);
            __syncthreads();
            n = s_cnt[bit];
            if (n >= left) {
                T = cand;
                above = n;
                if (n == left) break;  // exactly these
            }
        }
    }
    // `above` keys are >= T; of those equal to T the last `above - left` go
    // ---- ranks: ties (key == T), then free slots below left and kept ones past it
    auto each_strip = [&](auto &&body) {  // body(slot, in the request, key)
        if constexpr (KPT > 0) {
#pragma unroll
            for (int i = 0; i < KR; ++i)
                if (i < strips) body(s0 + 32 * i, s0 + 32 * i < L, key[i]);
        } else {
            for (int i = 0; i < strips; ++i) {
                const int s = s0 + 32 * i;
                body(s, s < L, s < L ? key_of(s) : 0u);
            }
        }
    };
    int ties = 0;
    each_strip([&](int, bool in, uint32_t kk) { ties += __popc(__ballot_sync(0xffffffffu, in && kk == T)); });
    if (lane == 0) s_warp[0][warp] = ties;
    __syncthreads();
    int all_ties = 0, ties_before = 0;
    for (int w = 0; w < NW; ++w) {
        const int t = s_warp[0][w];
        if (w < warp) ties_before += t;
        all_ties += t;
    }
    const int keep_ties = all_ties - (above - left);
    auto classify = [&](auto &&visit) {
        int tb = ties_before;
        each_strip([&](int s, bool in, uint32_t kk) {
            const unsigned tm = __ballot_sync(0xffffffffu, in && kk == T);
            const bool kept = in && (kk > T || (kk == T && tb + __popc(tm & ((1u << lane) - 1)) < keep_ties));
            tb += __popc(tm);
            const unsigned fm = __ballot_sync(0xffffffffu, in && !kept && s < left);
            const unsigned mm = __ballot_sync(0xffffffffu, kept && s >= left);
            visit(s, kept, in, fm, mm);
        });
    };
    int nfree = 0, nmove = 0;
    classify([&](int, bool, bool, unsigned fm, unsigned mm) {
        nfree += __popc(fm);
        nmove += __popc(mm);
    });
    if (lane == 0) {
        s_warp[1][warp] = nfree;
        s_warp[2][warp] = nmove;
    }
    __syncthreads();
    int f0 = 0, m0 = 0, moves = 0;
    for (int w = 0; w < NW; ++w) {
        if (w < warp) {
            f0 += s_warp[1][w];
            m0 += s_warp[2][w];
        }
        moves += s_warp[2][w];
    }
    int32_t *dst = P.lists + rowi * 2 * P.cap, *src = dst + P.cap;
    classify([&](int s, bool kept, bool in, unsigned fm, unsigned mm) {
        const unsigned lt = (1u << lane) - 1;
        if (in && s < left) {
            if (kept) {  // stays (its own entry: no other thread reads it)
                const int p = pos_of(s);
                mass_out[s] = mass[s];
                pos_out[s] = p;
            } else {
                dst[f0 + __popc(fm & lt)] = s;
            }
        } else if (kept) {
            src[m0 + __popc(mm & lt)] = s;
        }
        f0 += __popc(fm);
        m0 += __popc(mm);
    });
    __syncthreads();
    for (int i = tid; i < moves; i += THREADS) {
        const int s = src[i], d = dst[i];
        const float v = mass[s];
        const int p = pos_of(s);
        mass_out[d] = v;
        pos_out[d] = p;
    }
    __syncthreads();  // mass may be mass_out: the tail is cleared after its last read
    for (int s = left + tid; s < L; s += THREADS) mass_out[s] = 0.f;
    if (tid == 0) P.counts[rowi] = moves;
}

__global__ void __launch_bounds__(MOVE_THREADS) pa_evict_move_kernel(EvictParams P) {
    grid_dependency_wait();
    const int g = blockIdx.y % P.Hkv, b = blockIdx.y / P.Hkv;
    const size_t rowi = blockIdx.y;
    const int tid = threadIdx.x;
    if (blockIdx.x == 0 && g == 0 && tid == 0) {
        const int4 r = P.req[b];
        P.lens_out[b] = r.x;
        P.history_out[2 * b] = r.y;
        P.history_out[2 * b + 1] = r.z;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        uint32_t e = 0;
        for (int i = tid; i < P.B; i += MOVE_THREADS) e |= (uint32_t)P.req[i].w;
        e = __reduce_or_sync(0xffffffffu, e);
        __shared__ uint32_t s_e;
        if (tid == 0) s_e = 0;
        __syncthreads();
        if ((tid & 31) == 0 && e) atomicOr(&s_e, e);
        __syncthreads();
        if (tid == 0) P.hdr[0] = s_e;
    }
    const int n = P.counts[rowi], i0 = blockIdx.x * MOVE_ROWS;
    if (i0 >= n) return;
    const int rows = min(MOVE_ROWS, n - i0);
    const int32_t *dst = P.lists + rowi * 2 * P.cap + i0, *src = dst + P.cap;
    const int32_t *table = P.block_table + (size_t)b * P.tbl;
    __shared__ long long s_at[MOVE_ROWS][4];  // K source, K destination, V source, V destination
    if (tid < rows) {
        const int s = src[tid], d = dst[tid];
        const int bs_ = table[s / P.bs], bd = table[d / P.bs];
        const long long rs = (long long)g * P.bs + s % P.bs, rd = (long long)g * P.bs + d % P.bs;
        s_at[tid][0] = (long long)bs_ * P.k_block + rs * P.k_row;
        s_at[tid][1] = (long long)bd * P.k_block + rd * P.k_row;
        s_at[tid][2] = (long long)bs_ * P.v_block + rs * P.v_row;
        s_at[tid][3] = (long long)bd * P.v_block + rd * P.v_row;
        if (P.k_tok)
            *reinterpret_cast<float *>(P.k_pool + (long long)bd * P.k_block + P.k_codes + rd * 4) =
                *reinterpret_cast<const float *>(P.k_pool + (long long)bs_ * P.k_block + P.k_codes + rs * 4);
        if (P.v_tok)
            *reinterpret_cast<float *>(P.v_pool + (long long)bd * P.v_block + P.v_codes + rd * 4) =
                *reinterpret_cast<const float *>(P.v_pool + (long long)bs_ * P.v_block + P.v_codes + rs * 4);
    }
    __syncthreads();
    const int kp = P.k_row / 16, pieces = kp + P.v_row / 16, total = rows * pieces;
    constexpr int UN = 4;
    for (int base = tid; base < total; base += MOVE_THREADS * UN) {
        uint4 v[UN];
        uint4 *to[UN];
#pragma unroll
        for (int q = 0; q < UN; ++q) {
            const int i = base + q * MOVE_THREADS;
            if (i < total) {
                const int r = i / pieces, p = i - r * pieces;
                const bool isk = p < kp;
                uint8_t *pool = isk ? P.k_pool : P.v_pool;
                const int o = 16 * (isk ? p : p - kp);
                v[q] = *reinterpret_cast<const uint4 *>(pool + s_at[r][isk ? 0 : 2] + o);
                to[q] = reinterpret_cast<uint4 *>(pool + s_at[r][isk ? 1 : 3] + o);
            }
        }
#pragma unroll
        for (int q = 0; q < UN; ++q)
            if (base + q * MOVE_THREADS < total) *to[q] = v[q];
    }
}

}  // namespace evict
}  // namespace pa

namespace {

struct EvictLayout {
    size_t req, counts, lists, total;
    int cap;
};

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

pa_status evict_layout(const pa_problem *p, int32_t budget, EvictLayout *lo) {
    if (p == nullptr || lo == nullptr || p->batch < 0 || p->num_kv_heads < 1 || p->max_context_len < 0 || budget < 1)
        return PA_ERR_INVALID_ARG;
    if (p->max_context_len > (1 << 20) || (long long)p->batch * p->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
    // at most `budget` rows move, and at most the rows past it
    lo->cap = std::max(0, std::min(budget, p->max_context_len - budget));
    const size_t rows = (size_t)p->batch * p->num_kv_heads;
    lo->req = 256;
    lo->counts = lo->req + up256((size_t)p->batch * 16);
    lo->lists = lo->counts + up256(rows * 4);
    lo->total = lo->lists + up256(rows * 2 * lo->cap * 4);
    return PA_OK;
}

bool off_by(const void *x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) & (a - 1)) != 0; }

int bits_of(int dt) {
    switch (dt) {
        case PA_F16: case PA_BF16: return 16;
        case PA_E4M3: case PA_INT8: return 8;
        case PA_INT4: return 4;
        default: return 0;
    }
}

}  // namespace

extern "C" PA_API pa_status pa_evict_workspace_size(const pa_problem *p, int32_t budget, size_t *bytes) {
    if (bytes == nullptr) return PA_ERR_INVALID_ARG;
    EvictLayout lo;
    const pa_status st = evict_layout(p, budget, &lo);
    if (st != PA_OK) return st;
    *bytes = lo.total;
    return PA_OK;
}

extern "C" PA_API pa_status pa_evict(const pa_problem *p, int32_t budget, int32_t sinks, int32_t recent,
                                     const float *mass, const int32_t *positions, const int32_t *history,
                                     const int32_t *block_table, const int32_t *context_lens, void *k_pool,
                                     void *v_pool, float *mass_out, int32_t *positions_out, int32_t *history_out,
                                     int32_t *lens_out, void *workspace, size_t workspace_bytes, pa_stream_t stream) {
    EvictLayout lo;
    const pa_status st = evict_layout(p, budget, &lo);
    if (st != PA_OK) return st;
    if (sinks < 0 || recent < 0 || (long long)sinks + recent > budget || p->head_dim_k < 1 || p->head_dim_v < 1 ||
        p->block_size < 1 || p->num_blocks < 1 || p->max_blocks_per_seq < 1 || p->k_scale_mode < PA_SCALE_NONE ||
        p->k_scale_mode > PA_SCALE_TOKEN || p->v_scale_mode < PA_SCALE_NONE || p->v_scale_mode > PA_SCALE_TOKEN ||
        (p->v_is_k_prefix != 0 && p->v_is_k_prefix != 1))
        return PA_ERR_INVALID_ARG;
    const int bits = bits_of(p->kv_dtype);
    if (bits == 0) return PA_ERR_INVALID_ARG;
    const bool plane_v = p->v_is_k_prefix == 0;
    const long long kr = (long long)p->head_dim_k * bits, vr = plane_v ? (long long)p->head_dim_v * bits : 0;
    if (kr % 128 || vr % 128 || kr > (1 << 20) || vr > (1 << 20)) return PA_ERR_UNSUPPORTED;
    const long long slots = (long long)p->num_kv_heads * p->block_size;
    const long long kc = slots * (kr / 8), vc = slots * (vr / 8);
    const bool ktok = p->k_scale_mode == PA_SCALE_TOKEN, vtok = plane_v && p->v_scale_mode == PA_SCALE_TOKEN;
    const long long kb = kc + (ktok ? slots * 4 : 0), vb = vc + (vtok ? slots * 4 : 0);
    if (kb % 16 || vb % 16) return PA_ERR_UNSUPPORTED;
    if (workspace == nullptr || off_by(workspace, 256) || workspace_bytes < lo.total) return PA_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (p->batch == 0) return PA_OK;
    if (mass == nullptr || positions == nullptr || history == nullptr || block_table == nullptr ||
        context_lens == nullptr || k_pool == nullptr || (plane_v && v_pool == nullptr) || mass_out == nullptr ||
        positions_out == nullptr || history_out == nullptr || lens_out == nullptr)
        return PA_ERR_INVALID_ARG;
    if (off_by(mass, 4) || off_by(positions, 4) || off_by(history, 4) || off_by(block_table, 4) ||
        off_by(context_lens, 4) || off_by(k_pool, 16) || (plane_v && off_by(v_pool, 16)) || off_by(mass_out, 4) ||
        off_by(positions_out, 4) || off_by(history_out, 4) || off_by(lens_out, 4))
        return PA_ERR_INVALID_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    pa::EvictParams P;
    P.mass = mass;
    P.positions = positions;
    P.history = history;
    P.block_table = block_table;
    P.context_lens = context_lens;
    P.k_pool = static_cast<uint8_t *>(k_pool);
    P.v_pool = static_cast<uint8_t *>(v_pool);
    P.mass_out = mass_out;
    P.positions_out = positions_out;
    P.history_out = history_out;
    P.lens_out = lens_out;
    P.hdr = reinterpret_cast<uint32_t *>(ws);
    P.req = reinterpret_cast<int4 *>(ws + lo.req);
    P.counts = reinterpret_cast<int32_t *>(ws + lo.counts);
    P.lists = reinterpret_cast<int32_t *>(ws + lo.lists);
    P.k_block = kb;
    P.v_block = vb;
    P.k_codes = kc;
    P.v_codes = vc;
    P.k_row = (int)(kr / 8);
    P.v_row = (int)(vr / 8);
    P.k_tok = ktok;
    P.v_tok = vtok;
    P.B = p->batch;
    P.Hkv = p->num_kv_heads;
    P.bs = p->block_size;
    P.tbl = p->max_blocks_per_seq;
    P.max_ctx = p->max_context_len;
    P.num_blocks = p->num_blocks;
    P.budget = budget;
    P.sinks = sinks;
    P.recent = recent;
    P.cap = lo.cap;
    const dim3 grid((unsigned)p->num_kv_heads, (unsigned)p->batch);
    const int ctx = p->max_context_len, t = pa::evict::THREADS;
    if (ctx <= 8 * t) pa::evict::pa_evict_select_kernel<8><<<grid, t, 0, s>>>(P);
    else if (ctx <= 32 * t) pa::evict::pa_evict_select_kernel<32><<<grid, t, 0, s>>>(P);
    else pa::evict::pa_evict_select_kernel<0><<<grid, t, 0, s>>>(P);
    if (cudaPeekAtLastError() != cudaSuccess) return PA_ERR_CUDA;
    const unsigned chunks = (unsigned)std::max(1, (lo.cap + pa::evict::MOVE_ROWS - 1) / pa::evict::MOVE_ROWS);
    const cudaError_t e = pa::launch_pdl(pa::evict::pa_evict_move_kernel, dim3(chunks, (unsigned)(p->batch * p->num_kv_heads)),
                                         dim3(pa::evict::MOVE_THREADS), 0, s, P);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
