// Gradients of the permutation and of the weighted combine (steps 3 and 5; no
// counterpart on the source pages, which stop at the forward path):
//   combine   dy[r]   = bf16( w[t,j] * dout[t] ),  r = dest_row[t,j]
//             dw[t,j] = sum_h dout[t,h] * y[r,h]                   (fp32)
//             dl[t,e] = w[t,j] (dw[t,j] - sum_i w[t,i] dw[t,i]) at
//                       e = topk_idx[t,j], 0 elsewhere: the softmax over the
//                       selected logits, whose gradient is zero elsewhere
//   row copy  dx[t]   = bf16( sum_j dx_perm[dest_row[t,j]] ), fp32, slot order
// Both are gathers over a token's k rows, bound by HBM: every byte of y, dy
// (dx_perm) moves once and dout (dx) once per token, with 16-byte accesses.
// Nothing is accumulated with atomics, so results repeat bit for bit.
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
    int k, E, H8, P;
};

// One block per token.
__global__ void __launch_bounds__(kBwdThreads) k_combine_backward(CombineBwdArgs a) {
    __shared__ float part[kBwdThreads / 32][kBwdRows];
    __shared__ float s_dw[kMaxExperts];   // k <= E <= kMaxExperts
    __shared__ float s_row[kMaxExperts];  // the token's row of dlogits
    __shared__ float s_mean;
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    const uint4 *d = a.dout + (size_t)t * a.H8;
    for (int j0 = 0; j0 < a.k; j0 += kBwdRows) {
        int r[kBwdRows];
        float w[kBwdRows], acc[kBwdRows];
#pragma unroll
        for (int j = 0; j < kBwdRows; ++j) {
            const bool in = j0 + j < a.k;
            const int row = in ? __ldg(a.dest_row + (size_t)t * a.k + j0 + j) : -1;
            r[j] = (unsigned)row < (unsigned)a.P ? row : -1;
            w[j] = in ? __ldg(a.w + (size_t)t * a.k + j0 + j) : 0.0f;
            acc[j] = 0.0f;
        }
        for (int v = tid; v < a.H8; v += blockDim.x) {
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
#pragma unroll
        for (int j = 0; j < kBwdRows; ++j) {
#pragma unroll
            for (int off = 16; off; off >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], off);
            if (lane == 0) part[warp][j] = acc[j];
        }
        __syncthreads();
        if (tid < kBwdRows && j0 + tid < a.k) {
            float s = 0.0f;
            for (int i = 0; i < nw; ++i) s += part[i][tid];
            s_dw[j0 + tid] = s;
            a.dw[(size_t)t * a.k + j0 + tid] = s;
        }
        __syncthreads();
    }
    if (!a.dlogits) return;
    for (int e = tid; e < a.E; e += blockDim.x) s_row[e] = 0.0f;
    if (warp == 0) {
        float m = 0.0f;
        for (int j = lane; j < a.k; j += 32) m = fmaf(__ldg(a.w + (size_t)t * a.k + j), s_dw[j], m);
#pragma unroll
        for (int off = 16; off; off >>= 1) m += __shfl_xor_sync(0xffffffffu, m, off);
        if (lane == 0) s_mean = m;
    }
    __syncthreads();
    for (int j = tid; j < a.k; j += blockDim.x) {
        const int e = __ldg(a.topk_idx + (size_t)t * a.k + j);
        if ((unsigned)e < (unsigned)a.E) s_row[e] = __ldg(a.w + (size_t)t * a.k + j) * (s_dw[j] - s_mean);
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += blockDim.x) a.dlogits[(size_t)t * a.E + e] = s_row[e];
}

// Each thread owns 8 features of one token.
__global__ void __launch_bounds__(kBwdThreads)
    k_gather_backward(const uint4 *__restrict__ dx_perm, const int *__restrict__ dest_row, uint4 *__restrict__ dx, int k,
                      int H8, int P) {
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x;
    const int v = blockIdx.y * blockDim.x + threadIdx.x;
    if (v >= H8) return;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += kBwdRows) {
        uint4 q[kBwdRows];
        int r[kBwdRows];
#pragma unroll
        for (int j = 0; j < kBwdRows; ++j) r[j] = j0 + j < k ? __ldg(dest_row + (size_t)t * k + j0 + j) : -1;
#pragma unroll
        for (int j = 0; j < kBwdRows; ++j)
            q[j] = (unsigned)r[j] < (unsigned)P ? __ldg(dx_perm + (size_t)r[j] * H8 + v) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < kBwdRows; ++j) {
            if ((unsigned)r[j] >= (unsigned)P) continue;
            float f[8];
            unpack8f(q[j], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += f[i];
        }
    }
    dx[(size_t)t * H8 + v] = pack8f(acc);
}

int block_for(int H8) {
    const int t = (H8 + 31) / 32 * 32;
    return t < kBwdThreads ? t : kBwdThreads;
}

}  // namespace

cudaError_t launch_combine_backward(const moe_shape &s, const void *dout, const void *y, const int32_t *dest_row,
                                    const float *topk_w, const int32_t *topk_idx, void *dy, float *dtopk_w,
                                    float *dlogits, cudaStream_t stream) {
    CombineBwdArgs a = {};
    a.dout = (const uint4 *)dout;
    a.y = (const uint4 *)y;
    a.dest_row = dest_row;
    a.topk_idx = topk_idx;
    a.w = topk_w;
    a.dy = (uint4 *)dy;
    a.dw = dtopk_w;
    a.dlogits = dlogits;
    a.k = s.k;
    a.E = s.E;
    a.H8 = s.H / 8;
    a.P = (int)permuted_rows(s.T, s.E, s.k, s.C, (s.flags & MOE_FLAG_CAPACITY) != 0);
    return launch_pdl(k_combine_backward, dim3((unsigned)s.T), dim3((unsigned)block_for(a.H8)), 0, stream, a);
}

cudaError_t launch_gather_backward(const moe_shape &s, const void *dx_perm, const int32_t *dest_row, void *dx,
                                   cudaStream_t stream) {
    const int H8 = s.H / 8, bt = block_for(H8);
    const int P = (int)permuted_rows(s.T, s.E, s.k, s.C, (s.flags & MOE_FLAG_CAPACITY) != 0);
    return launch_pdl(k_gather_backward, dim3((unsigned)s.T, (unsigned)((H8 + bt - 1) / bt)), dim3((unsigned)bt), 0,
                      stream, (const uint4 *)dx_perm, dest_row, (uint4 *)dx, s.k, H8, P);
}

}  // namespace moe
