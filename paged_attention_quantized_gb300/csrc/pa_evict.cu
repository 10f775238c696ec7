// Eviction from the paged cache by accumulated attention weight.
//
// Selection (pa_evict_select_kernel), one CTA per (request, kv head): every
// slot gets a 32-bit key that orders as its mass does (protected slots the
// largest key, NaN the smallest), the left-th largest key is found digit by
// digit (11, 11, 10 bits) from histograms in shared memory until at most 32
// keys are left in question, which one warp then ranks; the slots above it plus
// the first of those equal to it are kept.  Keys stay in registers (up to 32
// slots per thread; longer rows read the mass again from L2 for every pass).
// The kept slots become a bitmap in shared memory, one ballot per 32 slots, and
// the number kept before each word comes from one scan: the rank of a free slot
// s below `left` is s less the kept ones before it, that of a kept slot at or
// past `left` is the kept ones between; the i-th of both pair up as the moves.
//
// Moves (pa_evict_move_kernel, or the selecting CTA when they are few): one thread per 16-byte piece of a moved K or V
// row.  Sources lie at or past `left`, destinations below it, so no row is
// read after it was written, whatever the order; HBM bound.
//
// Measured on a GB300: 512 rows of 2049-2064 tokens down to 2048 (a decode step)
// 14 us, all latency (about ten dependent steps of a microsecond); 128 rows of up
// to 16384 tokens, bf16 head dim 128, down to 2048 52 us (selection 20, moves 29 =
// 6 TB/s); 256 rows of up to 32768, E4M3 head dim 256, down to 4096 175 us
// (selection 58, two rounds of the SMs, moves 107 = 5.7 TB/s).  Finding the border
// key by 32 counted bits instead of digits took the last selection 89 us.
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

constexpr int MOVE_THREADS = 256, MOVE_ROWS = 128;  // rows of one CTA of the move kernel

// order-preserving key of a mass: larger mass, larger key; NaN below all (0)
__device__ __forceinline__ uint32_t mass_key(float v) {
    if (v != v) return 0u;
    const uint32_t u = __float_as_uint(v + 0.f);  // -0 counts as +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of v over the block's threads, and the total
template <int NW>
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t *s_warp, uint64_t &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const uint64_t t = s_warp[w];
        if (w < warp) before += t;
        all += t;
    }
    __syncthreads();
    total = all;
    return before + x - v;
}

// Rows i0 .. i0 + MOVE_ROWS - 1 of the moves of row `rowi` = (b, g), by THREADS
// threads; s_at: MOVE_ROWS x 4 entries of shared memory.  Sources lie at or past
// `left` and destinations below it, so the order does not matter.
template <int THREADS>
__device__ __forceinline__ void move_chunk(const EvictParams &P, int b, int g, size_t rowi, int i0, int n,
                                           long long (*s_at)[4]) {
    const int tid = threadIdx.x, rows = min(MOVE_ROWS, n - i0);
    const int32_t *dst = P.lists + rowi * 2 * P.cap + i0, *src = dst + P.cap;
    const int32_t *table = P.block_table + (size_t)b * P.tbl;
    for (int i = tid; i < rows; i += THREADS) {
        const int s = src[i], d = dst[i];
        const int bs_ = table[s / P.bs], bd = table[d / P.bs];
        const long long rs = (long long)g * P.bs + s % P.bs, rd = (long long)g * P.bs + d % P.bs;
        s_at[i][0] = (long long)bs_ * P.k_block + rs * P.k_row;
        s_at[i][1] = (long long)bd * P.k_block + rd * P.k_row;
        s_at[i][2] = (long long)bs_ * P.v_block + rs * P.v_row;
        s_at[i][3] = (long long)bd * P.v_block + rd * P.v_row;
        if (P.k_tok)
            *reinterpret_cast<float *>(P.k_pool + (long long)bd * P.k_block + P.k_codes + rd * 4) =
                *reinterpret_cast<const float *>(P.k_pool + (long long)bs_ * P.k_block + P.k_codes + rs * 4);
        if (P.v_tok)
            *reinterpret_cast<float *>(P.v_pool + (long long)bd * P.v_block + P.v_codes + rd * 4) =
                *reinterpret_cast<const float *>(P.v_pool + (long long)bs_ * P.v_block + P.v_codes + rs * 4);
    }
    __syncthreads();
    const int kp = P.k_row / 16, pieces = kp + P.v_row / 16;
    const int dr = THREADS / pieces, dp = THREADS - dr * pieces;
    int r = tid / pieces, p = tid - r * pieces;
    constexpr int UN = 4;
    while (r < rows) {
        uint4 v[UN];
        uint4 *to[UN];
#pragma unroll
        for (int q = 0; q < UN; ++q) {
            to[q] = nullptr;
            if (r < rows) {
                const bool isk = p < kp;
                uint8_t *pool = isk ? P.k_pool : P.v_pool;
                const int o = 16 * (isk ? p : p - kp);
                v[q] = *reinterpret_cast<const uint4 *>(pool + s_at[r][isk ? 0 : 2] + o);
                to[q] = reinterpret_cast<uint4 *>(pool + s_at[r][isk ? 1 : 3] + o);
            }
            r += dr;
            p += dp;
            if (p >= pieces) {
                p -= pieces;
                ++r;
            }
        }
#pragma unroll
        for (int q = 0; q < UN; ++q)
            if (to[q]) *to[q] = v[q];
    }
}

// Lengths and histories of the requests, and the error word
__device__ __forceinline__ void finish(const EvictParams &P) {
    __shared__ uint32_t s_e;
    if (threadIdx.x == 0) s_e = 0;
    __syncthreads();
    uint32_t e = 0;
    for (int b = threadIdx.x; b < P.B; b += blockDim.x) {
        const int4 r = P.req[b];
        P.lens_out[b] = r.x;
        P.history_out[2 * b] = r.y;
        P.history_out[2 * b + 1] = r.z;
        e |= (uint32_t)r.w;
    }
    if (e) atomicOr(&s_e, e);
    __syncthreads();
    if (threadIdx.x == 0) P.hdr[0] = s_e;
}

// KPT: slots per thread kept in registers (slot i * THREADS + thread), 0 = read again each time
// FUSED: the CTA moves its rows as well
template <int THREADS, int KPT, bool FUSED>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) pa_evict_select_kernel(EvictParams P) {
    constexpr int NW = THREADS / 32;
    grid_dependents_launch();  // the move kernel may queue up behind
    constexpr int BINS = 2048, BPT = BINS / THREADS;
    extern __shared__ uint32_t s_map[];  // one bit per slot, 32 consecutive slots a word; then the kept ones before each word
    __shared__ __align__(16) int s_hist[BINS];
    __shared__ int s_n, s_bin, s_over, s_in;
    static_assert(sizeof(s_hist) >= MOVE_ROWS * 32, "the moves' places use the histogram's room");
    __shared__ uint64_t s_warp[NW];
    __shared__ uint32_t s_few[32], s_pick, s_err;
    __shared__ int s_cut;
    grid_dependency_wait();
    const int g = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        s_n = 0;
        s_err = 0;
    }
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
    }
    const int left = min(L, P.budget);
    const size_t rowi = (size_t)b * P.Hkv + g;
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
    const int strips = err ? 0 : (L + THREADS - 1) / THREADS;  // slots of this thread: i * THREADS + tid, i < strips
    constexpr int KR = KPT > 0 ? KPT : 1;
    uint32_t key[KR];
    if constexpr (KPT > 0) {
        // loads first, eight of them in flight before the first is used
#pragma unroll
        for (int i0 = 0; i0 < KR; i0 += 8) {
            float v[8];
            int p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int s = (i0 + i) * THREADS + tid;
                v[i] = !err && s < L ? mass[s] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int s = (i0 + i) * THREADS + tid;
                p[i] = !err && s < base ? pos_in[s] : dropped + s;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool always = p[i] < P.sinks || p[i] >= newest;
                key[i0 + i] = err || (i0 + i) * THREADS + tid >= L ? 0u : always ? 0xFFFFFFFFu : mass_key(v[i]);
            }
        }
    }
    __syncthreads();
    if (err == 0) err = s_err;
    if (g == 0 && tid == 0)
        P.req[b] = err ? make_int4(L, base, dropped, (int)err) : make_int4(left, left, dropped + L - left, 0);
    if (err) {
        if (tid == 0) P.counts[rowi] = 0;
        return;
    }
    auto each = [&](auto &&body) {  // body(slot, in the request, key): whole warps, 32 consecutive slots each
        if constexpr (KPT > 0) {
#pragma unroll
            for (int i = 0; i < KR; ++i)
                if (i < strips) body(i * THREADS + tid, i * THREADS + tid < L, key[i]);
        } else {
            for (int i = 0; i < strips; ++i) {
                const int s = i * THREADS + tid;
                body(s, s < L, s < L ? key_of(s) : 0u);
            }
        }
    };
    // ---- the left-th largest key T: the largest T with at least `left` keys >= T
    uint32_t T = 0;
    int above = L, over = 0;  // keys >= T, keys past the interval in question
    for (int shift = 21; left < L; shift = max(0, shift - 11)) {
        // histogram of the keys of [T, T + 2^min(32, shift + 11)) by their next digit
        for (int i = tid; i < BINS; i += THREADS) s_hist[i] = 0;
        __syncthreads();
        each([&](int, bool in, uint32_t k) {
            const uint32_t d = (k - T) >> shift;
            const bool mine = in && k >= T && d < BINS;
            const unsigned m = __ballot_sync(0xffffffffu, mine);
            if (m == 0) return;
            const uint32_t d0 = __shfl_sync(0xffffffffu, d, __ffs(m) - 1);
            if (__all_sync(0xffffffffu, !mine || d == d0)) {  // (long runs of equal masses: one addition)
                if (lane == 0) atomicAdd(&s_hist[d0], __popc(m));
            } else if (mine) {
                atomicAdd(&s_hist[d], 1);
            }
        });
        __syncthreads();
        // the digit where the count from the top reaches `left`
        int c = 0;
#pragma unroll
        for (int i = 0; i < BPT; ++i) c += s_hist[BINS - 1 - (tid * BPT + i)];
        uint64_t total;
        int before = over + (int)block_scan<NW>((uint64_t)c, s_warp, total);
        if (before < left && left <= before + c) {
            for (int i = 0; i < BPT; ++i) {
                const int bin = BINS - 1 - (tid * BPT + i), h = s_hist[bin];
                if (left <= before + h) {
                    s_bin = bin;
                    s_over = before;
                    s_in = h;
                    break;
                }
                before += h;
            }
        }
        __syncthreads();
        T += (uint32_t)s_bin << shift;
        over = s_over;
        above = over + s_in;
        if (above == left || shift == 0) break;
        if (above - over <= 32) {
            // few keys are left in [T, T + 2^shift): list them, and rank them in one warp
            const uint32_t span = 1u << shift;
            each([&](int, bool in, uint32_t k) {
                if (in && k - T < span) s_few[atomicAdd(&s_n, 1)] = k;
            });
            __syncthreads();
            if (warp == 0) {
                const int m = above - over;
                const uint32_t k = lane < m ? s_few[lane] : 0u;
                int more = 0;  // keys at or above this lane's
                for (int i = 0; i < m; ++i) more += __shfl_sync(0xffffffffu, k, i) >= k ? 1 : 0;
                // the largest key with at least left - over of the few at or above it
                const bool ok = lane < m && over + more >= left;
                const uint32_t pick = __reduce_max_sync(0xffffffffu, ok ? k : T);
                if (ok && k == pick) {  // (equal keys agree)
                    s_pick = pick;
                    s_n = over + more;
                }
            }
            __syncthreads();
            T = s_pick;
            above = s_n;
            break;
        }
    }
    // ---- `above` keys are >= T; of those equal to T the last above - left in slot order go:
    // the ones from slot s_cut on
    const int words = (L + 31) / 32, wpt = (words + THREADS - 1) / THREADS;
    const int w0 = min(words, tid * wpt), w1 = min(words, w0 + wpt);  // this thread's words in the scans
    if (tid == 0) s_cut = L;
    if (above > left) {
        each([&](int s, bool in, uint32_t k) {
            const unsigned m = __ballot_sync(0xffffffffu, in && k == T);
            if (lane == 0 && in) s_map[s >> 5] = m;
        });
        __syncthreads();
        int n = 0;
        for (int w = w0; w < w1; ++w) n += __popc(s_map[w]);
        uint64_t total;
        int before = (int)block_scan<NW>((uint64_t)n, s_warp, total);
        const int keep = (int)total - (above - left);  // ties that stay
        if (before < keep + 1 && keep < before + n) {   // the first one to go is among this thread's words
            for (int w = w0; w < w1; ++w) {
                unsigned m = s_map[w];
                const int c = __popc(m);
                if (keep < before + c) {
                    for (int i = before; i < keep; ++i) m &= m - 1;
                    s_cut = w * 32 + __ffs(m) - 1;
                    break;
                }
                before += c;
            }
        }
        __syncthreads();
    }
    __syncthreads();
    const int cut = s_cut;
    each([&](int s, bool in, uint32_t k) {
        const unsigned m = __ballot_sync(0xffffffffu, in && (k > T || (k == T && s < cut)));
        if (lane == 0 && in) s_map[s >> 5] = m;
    });
    __syncthreads();
    // ---- how many are kept before each word, and below left
    uint32_t *s_before = s_map + words;
    int n = 0;
    for (int w = w0; w < w1; ++w) n += __popc(s_map[w]);
    uint64_t total;
    int at = (int)block_scan<NW>((uint64_t)n, s_warp, total);
    for (int w = w0; w < w1; ++w) {
        s_before[w] = at;
        at += __popc(s_map[w]);
    }
    __syncthreads();
    auto kept_before = [&](int s) -> int {  // of slots below s, s < 32 * words
        return (int)s_before[s >> 5] + __popc(s_map[s >> 5] & ((1u << (s & 31)) - 1));
    };
    const int stay = left < L ? kept_before(left) : left, moves = left - stay;
    int32_t *dst = P.lists + rowi * 2 * P.cap, *src = dst + P.cap;
    // ---- the kept slots below left keep their entries (their own: no other
    // thread reads them), the free ones and the kept ones past left are listed
#pragma unroll 4
    for (int s = tid; s < left; s += THREADS) {
        if ((s_map[s >> 5] >> (s & 31)) & 1u) {
            const int p = pos_of(s);
            mass_out[s] = mass[s];
            pos_out[s] = p;
        } else {
            dst[s - kept_before(s)] = s;
        }
    }
#pragma unroll 4
    for (int s = left + tid; s < L; s += THREADS)
        if ((s_map[s >> 5] >> (s & 31)) & 1u) src[kept_before(s) - stay] = s;
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
    if constexpr (FUSED) {
        for (int i0 = 0; i0 < moves; i0 += MOVE_ROWS) {
            move_chunk<THREADS>(P, b, g, rowi, i0, moves, reinterpret_cast<long long (*)[4]>(s_hist));
            __syncthreads();
        }
    } else {
        if (tid == 0) P.counts[rowi] = moves;
    }
}

__global__ void __launch_bounds__(MOVE_THREADS) pa_evict_move_kernel(EvictParams P) {
    __shared__ long long s_at[MOVE_ROWS][4];  // K source, K destination, V source, V destination
    grid_dependents_launch();
    grid_dependency_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0) finish(P);
    const size_t rowi = blockIdx.y;
    const int n = P.counts[rowi], i0 = blockIdx.x * MOVE_ROWS;
    if (i0 < n) move_chunk<MOVE_THREADS>(P, blockIdx.y / P.Hkv, blockIdx.y % P.Hkv, rowi, i0, n, s_at);
}

__global__ void __launch_bounds__(MOVE_THREADS) pa_evict_finish_kernel(EvictParams P) {
    grid_dependents_launch();
    grid_dependency_wait();
    finish(P);
}

template <bool FUSED>
cudaError_t launch_select(const EvictParams &P, dim3 grid, size_t map, cudaStream_t s) {
    const int ctx = P.max_ctx;
    if (ctx <= 4096) return launch_pdl(pa_evict_select_kernel<256, 16, FUSED>, grid, dim3(256), map, s, P);
    if (ctx <= 16384) return launch_pdl(pa_evict_select_kernel<1024, 16, FUSED>, grid, dim3(1024), map, s, P);
    if (ctx <= 32768) return launch_pdl(pa_evict_select_kernel<1024, 32, FUSED>, grid, dim3(1024), map, s, P);
    if (map > 36 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(pa_evict_select_kernel<1024, 0, FUSED>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (1 << 17) + 16);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(pa_evict_select_kernel<1024, 0, FUSED>, grid, dim3(1024), map, s, P);
}

}  // namespace evict
}  // namespace pa

namespace {

constexpr int MAX_CONTEXT = 1 << 19;  // the select kernel's bitmap and counts: 128 KB of shared memory

struct EvictLayout {
    size_t req, counts, lists, total;
    int cap;
};

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

pa_status evict_layout(const pa_problem *p, int32_t budget, EvictLayout *lo) {
    if (p == nullptr || lo == nullptr || p->batch < 0 || p->num_kv_heads < 1 || p->max_context_len < 0 || budget < 1)
        return PA_ERR_INVALID_ARG;
    if (p->max_context_len > MAX_CONTEXT || (long long)p->batch * p->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
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
    const size_t map = ((size_t)p->max_context_len + 31) / 32 * 8 + 16;  // the bitmap of kept slots, the counts before its words
    // The CTA that selected moves its rows itself while they are one chunk at most (a
    // decode step: 512 rows of 2064 tokens down to 2048, 14.5 us; 16.4 with a move
    // kernel); with more, a kernel over all SMs does (128 rows of up to 16384 down to
    // 2048: 55 us; 68 fused, since a CTA's chunks wait for one another).
    const bool fused = lo.cap <= pa::evict::MOVE_ROWS;
    cudaError_t e = fused ? pa::evict::launch_select<true>(P, grid, map, s) : pa::evict::launch_select<false>(P, grid, map, s);
    if (e != cudaSuccess) return PA_ERR_CUDA;
    if (fused) {
        e = pa::launch_pdl(pa::evict::pa_evict_finish_kernel, dim3(1), dim3(pa::evict::MOVE_THREADS), 0, s, P);
    } else {
        const unsigned chunks = (unsigned)std::max(1, (lo.cap + pa::evict::MOVE_ROWS - 1) / pa::evict::MOVE_ROWS);
        e = pa::launch_pdl(pa::evict::pa_evict_move_kernel, dim3(chunks, (unsigned)(p->batch * p->num_kv_heads)),
                           dim3(pa::evict::MOVE_THREADS), 0, s, P);
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
