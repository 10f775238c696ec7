// Shared by the two kernels of the accumulated attention weight (pa_mass.cu,
// pa_mass_tc.cu): parameters, the operand order of decoded codes, and the
// prefix sum of the requests' units of work.
#pragma once

#include "pa_attn.cuh"

namespace pa {

struct MassParams {
    const uint8_t *q;
    const uint8_t *k_pool;
    const int32_t *block_table;
    const int32_t *context_lens;
    const float *k_scale;
    const float *lse;
    float *mass;
    uint32_t *dev_error;
    long long k_block;   // bytes per pool block
    int k_codes;         // bytes of codes in a block (the per-token scales follow)
    int B, n, Hq, Hkv, G, R, bs, tbl, max_ctx, num_blocks;
    int q_dtype, k_mode, causal;
    unsigned bs_mul;     // floor(2^32 / bs) + 1: token / bs is the high word of the product (tokens * bs < 2^32)
    float decay, softmax_scale;
};

namespace mass {

constexpr int MAX_B = 4096;

__device__ __forceinline__ float q_val(const uint8_t *row, int ch, int dtype) {
    const uint16_t u = reinterpret_cast<const uint16_t *>(row)[ch];
    return dtype == PA_BF16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}

// the channel of element e (0, 1) of operand word w (0 ..) of 16-byte piece
// `piece` of a row of BITS-bit codes
template <int BITS>
__device__ __forceinline__ int channel_of(int piece, int w, int e) {
    if (BITS == 16) return piece * 8 + 2 * w + e;
    if (BITS == 8) return piece * 16 + 2 * w + e;
    return piece * 32 + 8 * (w >> 2) + (w & 3) + 4 * e;  // nibbles k and k + 4 of a 32-bit word
}

// one 16-byte piece of codes -> its operand words (f16x2 or bf16x2)
template <int KV>
__device__ __forceinline__ void decode(uint4 v, uint32_t *w) {
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (KV == PA_F16 || KV == PA_BF16) {
            w[i] = in[i];
        } else if constexpr (KV == PA_E4M3) {
            w[2 * i] = e4m3x2_f16x2(in[i]);
            w[2 * i + 1] = e4m3x2_f16x2(in[i] >> 16);
        } else if constexpr (KV == PA_INT8) {
            const uint32_t u = in[i] ^ 0x80808080u;
            w[2 * i] = u8pair_f16x2(u, 0x4140);
            w[2 * i + 1] = u8pair_f16x2(u, 0x4342);
        } else {
            w[4 * i] = s4lo_f16x2(in[i]);
            w[4 * i + 1] = s4hi_f16x2(in[i]);
            w[4 * i + 2] = s4lo_f16x2(in[i] >> 8);
            w[4 * i + 3] = s4hi_f16x2(in[i] >> 8);
        }
    }
}

// Prefix sums ps[0 .. B] (shared memory) of the requests' units of UT tokens,
// by all NT threads of the CTA; a request whose length breaks the contract
// has none.  Returns whether this thread saw such a request.
template <int NT, int UT>
__device__ __forceinline__ bool scan_units(const MassParams &P, int *ps, int *warp_tot) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int carry = 0;
    bool bad = false;
    for (int base = 0; base < P.B; base += NT) {
        const int b = base + tid;
        int u = 0;
        if (b < P.B) {
            const int L = P.context_lens[b];
            if (L < 0 || L > P.max_ctx || (long long)L > (long long)P.tbl * P.bs) bad = true;
            else u = (L + UT - 1) / UT;
        }
        int x = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_tot[warp] = x;
        __syncthreads();
        int before = carry, all = 0;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
            const int t = warp_tot[i];
            if (i < warp) before += t;
            all += t;
        }
        if (b < P.B) ps[b] = before + x - u;
        carry += all;
        __syncthreads();
    }
    if (tid == 0) ps[P.B] = carry;
    __syncthreads();
    return bad;
}

// the request that unit position u0 (over one kv head) belongs to
__device__ __forceinline__ int request_of(const int *ps, int B, int u0) {
    int lo = 0, hi = B;  // ps[lo] <= u0 < ps[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ps[mid] <= u0) lo = mid;
        else hi = mid;
    }
    return lo;
}

cudaError_t launch_mass_tc(const MassParams &P, int kv, int D, int nt, int sms, cudaStream_t s);

}  // namespace mass
}  // namespace pa
