// Drafted tokens (a tree of them, or a plain run) over a paged cache, head
// dim 512, sm_103a.
//
// With start = len - cnt the last cnt cached positions are the tokens' own.
// Token t sees a key j < start always and a key start + c if its mask has bit
// c (no mask: c <= t); with a window, only keys whose place is above the
// token's place - window or below n_sinks, where the place of a cached key is
// its position and that of token t is start + (tokens it sees) - 1.
//
// One block per (head, token, sequence): its warps stride over the keys, each
// with its own online softmax, and merge at the end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fa512_device.cuh"
#include "fa512_internal.h"

namespace fa512 {
namespace tree {

constexpr int D = 512;
constexpr int MAX_NODES = 256;
constexpr int WARPS = 8;

__device__ __forceinline__ void widen8(const uint4 a, float* f) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void widen16_e4m3(const uint4 a, float* f) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const unsigned short two = static_cast<unsigned short>(w[i >> 1] >> (16 * (i & 1)));
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
        asm("cvt.f32.f16 %0, %1;" : "=f"(f[2 * i]) : "h"(static_cast<unsigned short>(h2 & 0xffffu)));
        asm("cvt.f32.f16 %0, %1;" : "=f"(f[2 * i + 1]) : "h"(static_cast<unsigned short>(h2 >> 16)));
    }
}

// This lane's 16 columns of a cached row.
template <bool FP8>
__device__ __forceinline__ void load16(const void* pages, size_t row, int lane, float* f) {
    if constexpr (FP8) {
        widen16_e4m3(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pages) + row * D)[lane], f);
    } else {
        const uint4* r = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pages) + row * D);
        widen8(r[2 * lane], f);
        widen8(r[2 * lane + 1], f + 8);
    }
}

template <bool FP8>
__global__ void __launch_bounds__(WARPS * 32) tree_rows_kernel(const TreeParams p) {
    __shared__ float so[WARPS][D];
    __shared__ float sm[WARPS], sl[WARPS];
    __shared__ int depth[MAX_NODES];
    const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int len = p.kv_lens[b], cnt = p.q_lens ? p.q_lens[b] : p.q_len;
    if (len < 0 || len > p.len_cap || cnt < 0 || cnt > p.q_len) {
        if (threadIdx.x == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        len = len < 0 ? 0 : min(len, p.len_cap);
        cnt = cnt < 0 ? 0 : min(cnt, p.q_len);
    }
    const int start = len - cnt;
    const bool real = t < cnt && start + t >= 0;
    auto sees = [&](int a, int c) {
        return p.tree_mask ? (p.tree_mask[(static_cast<size_t>(b) * p.q_len + a) * p.mask_words + (c >> 5)] >> (c & 31)) & 1
                           : c <= a;
    };
    if (p.tree_mask)
        for (int a = threadIdx.x; a < cnt; a += WARPS * 32) {
            int n = 0;
            for (int c = 0; c < cnt; ++c) n += sees(a, c);
            depth[a] = n - 1;
        }
    __syncthreads();
    const int place = start + (real && p.tree_mask ? depth[t] : t);

    float q[16], o[16], m = -INFINITY, l = 0.f;
    const size_t row_q = (static_cast<size_t>(b) * p.q_len + t) * p.n_q_heads + h;
    widen8(reinterpret_cast<const uint4*>(p.q + row_q * D)[2 * lane], q);
    widen8(reinterpret_cast<const uint4*>(p.q + row_q * D)[2 * lane + 1], q + 8);
#pragma unroll
    for (int d = 0; d < 16; ++d) o[d] = 0.f;
    const int kvh = h / p.group;
    // keys below the window's first place, other than the sinks, are skipped
    const int lo = p.window > 0 ? max(0, min(place, start) - p.window + 1) : 0;
    const int skip_from = min(p.n_sinks, lo);
    if (real)
        for (int i = warp; i < skip_from + len - lo; i += WARPS) {
            const int j = i < skip_from ? i : lo + i - skip_from;
            const int c = j - start;
            if (c >= 0 && !sees(t, c)) continue;
            const int kp = c < 0 ? j : start + (p.tree_mask ? depth[c] : c);
            if (p.window > 0 && kp <= place - p.window && kp >= p.n_sinks) continue;
            const int page = p.page_table[static_cast<size_t>(b) * p.max_pages_per_seq + j / p.page_size];
            if (page < 0 || page >= p.num_pages) {
                if (lane == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
                continue;
            }
            const size_t row = (static_cast<size_t>(page) * p.page_size + j % p.page_size) * p.n_kv_heads + kvh;
            float f[16], s = 0.f;
            load16<FP8>(p.k_pages, row, lane, f);
#pragma unroll
            for (int d = 0; d < 16; ++d) s = fmaf(q[d], f[d], s);
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            s *= p.scale_log2;
            const float mn = fmaxf(m, s);
            const float a = fast_exp2(m - mn), e = fast_exp2(s - mn);
            m = mn;
            l = l * a + e;
            load16<FP8>(p.v_pages, row, lane, f);
#pragma unroll
            for (int d = 0; d < 16; ++d) o[d] = fmaf(e, f[d], o[d] * a);
        }
#pragma unroll
    for (int d = 0; d < 16; ++d) so[warp][lane * 16 + d] = o[d];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm[w]);
    float wt[WARPS];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        wt[w] = M == -INFINITY ? 0.f : fast_exp2(sm[w] - M);
        L += wt[w] * sl[w];
    }
    const float inv = L > 0.f ? p.o_scale / L : 0.f;
    for (int d = threadIdx.x; d < D; d += WARPS * 32) {
        float acc = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            if (wt[w] != 0.f) acc = fmaf(wt[w], so[w][d], acc);
        p.out[row_q * D + d] = __float2bfloat16_rn(M == -INFINITY ? 0.f : acc * inv);
    }
    if (p.lse && threadIdx.x == 0)
        p.lse[row_q] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

}  // namespace tree

int tree_max_nodes() { return tree::MAX_NODES; }

cudaError_t launch_decode_tree(const TreeParams& p, bool fp8, cudaStream_t stream) {
    const dim3 grid(p.n_q_heads, p.q_len, p.batch);
    if (fp8)
        tree::tree_rows_kernel<true><<<grid, tree::WARPS * 32, 0, stream>>>(p);
    else
        tree::tree_rows_kernel<false><<<grid, tree::WARPS * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fa512
