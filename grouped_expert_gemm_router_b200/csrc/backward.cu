// Gradients of the permutation and of the weighted combine (steps 3 and 5; no
// counterpart on the source pages, which stop at the forward path):
//   combine   dy[r]   = bf16( w[t,j] * dout[t] ),  r = dest_row[t,j]
//             dw[t,j] = sum_h dout[t,h] * y[r,h]                   (fp32)
//             dl[t,e] = w[t,j] (dw[t,j] - sum_i w[t,i] dw[t,i]) at
//                       e = topk_idx[t,j], 0 elsewhere: the softmax over the
//                       selected logits, whose gradient is zero elsewhere
//   row copy  dx[t]   = bf16( sum_j dx_perm[dest_row[t,j]] ), fp32, slot order
// Both are gathers over a token's k rows, bound by HBM: every byte of y, dy
// (dx_perm) moves once and dout (dx) once per token, with 16-byte accesses and
// about eight of them in flight per thread (8192 tokens: combine, 2048
// features, k 8: 97 us, 5.9 TB/s; row copy, 4096 features, k 2: 37 us, 5.4
// TB/s).  Nothing is accumulated with atomics, so results repeat bit for bit.
#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {

namespace {

constexpr int kBwdThreads = 256;
constexpr int kBwdRows = 8;  // rows of a token handled per pass

__device__ __forceinline__ void unpack8f(const uint4 &q, float (&v)[8]) {
    const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(b[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8f(const float (&v)[8]) {
    uint4 o;
    __nv_bfloat162 *b = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    return o;
}

struct CombineBwdArgs {
    const uint4 *dout, *y;
    const int *dest_row, *topk_idx;
    const float *w;
    uint4 *dy;
    float *dw, *dlogits;
    int T, k, E, H8, P;
};

// Sums the kBwdRows values of all 32 lanes: afterwards every lane holds the
// total of value (lane & 7).  Each step halves the values a lane carries, so
// eight sums take 9 shuffles instead of 40.
__device__ __forceinline__ float warp_sum8(const float (&v)[kBwdRows], int lane) {
    float a[4], b[2], c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // lanes with bit 2 take values 4-7
        const float mine = lane & 4 ? v[i + 4] : v[i], other = lane & 4 ? v[i] : v[i + 4];
        a[i] = mine + __shfl_xor_sync(0xffffffffu, other, 4);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float mine = lane & 2 ? a[i + 2] : a[i], other = lane & 2 ? a[i] : a[i + 2];
        b[i] = mine + __shfl_xor_sync(0xffffffffu, other, 2);
    }
    const float mine = lane & 1 ? b[1] : b[0], other = lane & 1 ? b[0] : b[1];
    c = mine + __shfl_xor_sync(0xffffffffu, other, 1);
    c += __shfl_xor_sync(0xffffffffu, c, 8);
    c += __shfl_xor_sync(0xffffffffu, c, 16);
    return c;
}

// W warps per token, 8 / W tokens per block.  The dot products need a token's
// whole row, so the fewer warps share a token the less is exchanged; more
// warps per token only where there are too few tokens to fill the SMs.
template <int W>
__global__ void __launch_bounds__(kBwdThreads, 3) k_combine_backward(CombineBwdArgs a) {
    constexpr int kTok = 8 / W;
    __shared__ float part[8][kBwdRows];
    __shared__ float s_dw[kTok][kMaxExperts];   // k <= E <= kMaxExperts
    __shared__ float s_row[kTok][kMaxExperts];  // the token's row of dlogits
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slot = warp / W, tw = (warp % W) * 32 + lane;  // token of the block, thread of the token
    const int t = blockIdx.x * kTok + slot;
    const bool live = t < a.T;
    const uint4 *d = a.dout + (size_t)t * a.H8;
    auto sync = [&]() {
        if (W == 1) __syncwarp();
        else __syncthreads();
    };
    for (int j0 = 0; j0 < a.k; j0 += kBwdRows) {
        int r[kBwdRows];
        float w[kBwdRows], acc[kBwdRows];
#pragma unroll
        for (int j = 0; j < kBwdRows; ++j) {
            const bool in = live && j0 + j < a.k;
            const int row = in ? __ldg(a.dest_row + (size_t)t * a.k + j0 + j) : -1;
            r[j] = (unsigned)row < (unsigned)a.P ? row : -1;
            w[j] = in ? __ldg(a.w + (size_t)t * a.k + j0 + j) : 0.0f;
            acc[j] = 0.0f;
        }
        if (live) {
            for (int v = tw; v < a.H8; v += 32 * W) {
                uint4 q[kBwdRows];
                const uint4 dq = __ldg(d + v);
#pragma unroll
                for (int j = 0; j < kBwdRows; ++j)
                    q[j] = r[j] >= 0 ? __ldg(a.y + (size_t)r[j] * a.H8 + v) : make_uint4(0, 0, 0, 0);
                float df[8];
                unpack8f(dq, df);
#pragma unroll
                for (int j = 0; j < kBwdRows; ++j) {
                    if (r[j] < 0) continue;
                    float yf[8], o[8];
                    unpack8f(q[j], yf);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        acc[j] = fmaf(df[i], yf[i], acc[j]);
                        o[i] = w[j] * df[i];
                    }
                    a.dy[(size_t)r[j] * a.H8 + v] = pack8f(o);
                }
            }
        }
        float s = warp_sum8(acc, lane);
        if (W > 1) {
            if (lane < kBwdRows) part[warp][lane] = s;
            sync();
            if (tw < kBwdRows) {
                s = 0.0f;
                for (int i = 0; i < W; ++i) s += part[slot * W + i][tw];
            }
        }
        if (live && tw < kBwdRows && j0 + tw < a.k) {
            s_dw[slot][j0 + tw] = s;
            a.dw[(size_t)t * a.k + j0 + tw] = s;
        }
        sync();
    }
    if (!a.dlogits) return;
    for (int e = tw; e < a.E; e += 32 * W) s_row[slot][e] = 0.0f;
    // every warp of the token: sum_i w_i dw_i
    float m = 0.0f;
    if (live)
        for (int j = lane; j < a.k; j += 32) m = fmaf(__ldg(a.w + (size_t)t * a.k + j), s_dw[slot][j], m);
#pragma unroll
    for (int off = 16; off; off >>= 1) m += __shfl_xor_sync(0xffffffffu, m, off);
    sync();
    if (live) {
        for (int j = tw; j < a.k; j += 32 * W) {
            const int e = __ldg(a.topk_idx + (size_t)t * a.k + j);
            if ((unsigned)e < (unsigned)a.E)
                s_row[slot][e] = __ldg(a.w + (size_t)t * a.k + j) * (s_dw[slot][j] - m);
        }
    }
    sync();
    if (live)
        for (int e = tw; e < a.E; e += 32 * W) a.dlogits[(size_t)t * a.E + e] = s_row[slot][e];
}

// Each thread owns 8 features of NT tokens of at most KM rows each (KM = 0:
// one token, any number of rows, eight at a time), all their row loads in
// flight at once.
template <int KM, int NT>
__global__ void __launch_bounds__(kBwdThreads)
    k_gather_backward(const uint4 *__restrict__ dx_perm, const int *__restrict__ dest_row, uint4 *__restrict__ dx, int T,
                      int k, int H8, int P) {
    constexpr int K = KM ? KM : kBwdRows;
    pdl_trigger();
    pdl_wait();
    const int t0 = blockIdx.x * NT;
    const int v = blockIdx.y * blockDim.x + threadIdx.x;
    if (v >= H8) return;
    float acc[NT][8];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[n][i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += K) {
        uint4 q[NT][K];
        int r[NT][K];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < K; ++j)
                r[n][j] = t0 + n < T && j0 + j < k ? __ldg(dest_row + (size_t)(t0 + n) * k + j0 + j) : -1;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < K; ++j)
                q[n][j] = (unsigned)r[n][j] < (unsigned)P ? __ldcs(dx_perm + (size_t)r[n][j] * H8 + v)
                                                          : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < K; ++j) {
                float f[8];
                unpack8f(q[n][j], f);  // a skipped row adds zeros
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[n][i] += f[i];
            }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
        if (t0 + n < T) dx[(size_t)(t0 + n) * H8 + v] = pack8f(acc[n]);
}

int block_for(int H8) {
    const int t = (H8 + 31) / 32 * 32;
    return t < kBwdThreads ? t : kBwdThreads;
}

}  // namespace

cudaError_t launch_combine_backward(const moe_shape &s, const void *dout, const void *y, const int32_t *dest_row,
                                    const float *topk_w, const int32_t *topk_idx, void *dy, float *dtopk_w,
                                    float *dlogits, int num_sms, cudaStream_t stream) {
    CombineBwdArgs a = {};
    a.dout = (const uint4 *)dout;
    a.y = (const uint4 *)y;
    a.dest_row = dest_row;
    a.topk_idx = topk_idx;
    a.w = topk_w;
    a.dy = (uint4 *)dy;
    a.dw = dtopk_w;
    a.dlogits = dlogits;
    a.T = s.T;
    a.k = s.k;
    a.E = s.E;
    a.H8 = s.H / 8;
    a.P = (int)permuted_rows(s.T, s.E, s.k, s.C, (s.flags & MOE_FLAG_CAPACITY) != 0);
    // One warp per token once that gives every SM its three blocks of eight
    // warps (8192 tokens of 2048 features, k 8: 97 us against 106 with four
    // warps per token and 125 with eight); below that a token's row is shared,
    // as far as it has work for the warps (32 features a lane).
    auto go = [&](auto kernel, int tokens) {
        return launch_pdl(kernel, dim3((unsigned)((s.T + tokens - 1) / tokens)), dim3(kBwdThreads), 0, stream, a);
    };
    const int64_t full = 3ll * num_sms;
    if (s.T >= 8 * full || s.H <= 256) return go(k_combine_backward<1>, 8);
    if (s.T >= 2 * full || s.H <= 1024) return go(k_combine_backward<4>, 2);
    return go(k_combine_backward<8>, 1);
}

cudaError_t launch_gather_backward(const moe_shape &s, const void *dx_perm, const int32_t *dest_row, void *dx,
                                   cudaStream_t stream) {
    const int H8 = s.H / 8, bt = block_for(H8);
    const int P = (int)permuted_rows(s.T, s.E, s.k, s.C, (s.flags & MOE_FLAG_CAPACITY) != 0);
    const unsigned gy = (unsigned)((H8 + bt - 1) / bt);
    auto go = [&](auto kernel, int nt) {
        return launch_pdl(kernel, dim3((unsigned)((s.T + nt - 1) / nt), gy), dim3((unsigned)bt), 0, stream,
                          (const uint4 *)dx_perm, dest_row, (uint4 *)dx, s.T, s.k, H8, P);
    };
    // Eight row loads in flight per thread (8192 tokens, k 2: 37 us against 58
    // with one token per thread).  dx_perm is read once and not kept in L2
    // (37 us against 40).
    if (s.k == 1) return go(k_gather_backward<1, 8>, 8);
    if (s.k == 2) return go(k_gather_backward<2, 4>, 4);
    if (s.k <= 4) return go(k_gather_backward<4, 2>, 2);
    return go(k_gather_backward<0, 1>, 1);
}

}  // namespace moe
