// kv_attention.hip -- attention over the paged cache.
//
// The simplest form: one workgroup per (row, query head), a chunk of 256
// positions at a time: scores, the running maximum and sum, then the weighted
// sum of the values.
#include "kv_device.h"

namespace moe {

template <int D, int BITS>
__global__ __launch_bounds__(256) void k_attn_row(KvArgs a, const uint16_t *q, int64_t q_stride, void *out,
                                                  int out_f32, float *lse)
{
    __shared__ float qs[D], w[256], red[4], acc4[256];
    const int tid = threadIdx.x, h = blockIdx.y, i = blockIdx.x % a.max_rows, s = blockIdx.x / a.max_rows;
    const KvSeq sq = kv_seq(a, s);
    if (i >= sq.n) return;
    const int row = sq.row0 + i, p = sq.len - sq.n_pos + i, L = kv_limit(a, sq), P = 1 << a.page_log2;
    const int kh = h / (a.q_heads / a.kv_heads);
    const int hi = a.causal ? min(L, p + 1) : L, lo = a.window ? max(0, p - a.window + 1) : 0;
    const int slot = BITS == 8 ? kv_slot(a, s) : -1;
    if (tid < D) qs[tid] = bf16_to_f32(q[row * q_stride + h * D + tid]) * a.scale;
    __syncthreads();
    float m = -INFINITY, l = 0.f, acc = 0.f;  // acc: value tid % D over a share of the positions
    constexpr int SH = 256 / D;
    auto block_of = [&](int j, const uint16_t *&half, const uint16_t *&vhalf, int64_t &id) {
        const int pg = j >> a.page_log2;
        id = kv_page(a, s, pg);
        half = vhalf = nullptr;
        if (id < 0) return false;
        if (BITS == 16) {
            half = (const uint16_t *)a.k + kv_block_at(a, id, kh);
            vhalf = (const uint16_t *)a.v + kv_block_at(a, id, kh);
        } else if (((pg + 1) << a.page_log2) > L) {
            if (slot < 0) return false;
            const int64_t at = kv_block_at(a, (int64_t)slot * 2 + (pg & 1), kh);
            half = a.k_tail + at;
            vhalf = a.v_tail + at;
        }
        return true;
    };
    for (int c = lo; c < hi; c += 256) {
        const int j = c + tid;
        float z = -INFINITY;
        const uint16_t *half, *vhalf;
        int64_t id;
        if (j < hi && block_of(j, half, vhalf, id)) {
            z = 0.f;
            const int r = j & (P - 1);
            if (half) {
                for (int d = 0; d < D; ++d) z += qs[d] * bf16_to_f32(half[r * D + d]);
            } else {
                const int8_t *kc = (const int8_t *)a.k + kv_block_at(a, id, kh) + r * D;
                for (int d = 0; d < D; ++d) z += qs[d] * (float)kc[d];
                z *= a.k_scale[id * a.kv_heads + kh];
            }
        }
        float mx = z;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, WAVE));
        if ((tid & 63) == 0) red[tid >> 6] = mx;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float base = mn > -INFINITY ? mn : 0.f;
        const float e = z > -INFINITY || z != z ? __expf(z - base) : 0.f, f = m > -INFINITY ? __expf(m - base) : 0.f;
        w[tid] = e;
        __syncthreads();
        float sum = e;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, WAVE);
        if ((tid & 63) == 0) red[tid >> 6] = sum;
        acc *= f;
        const int d = tid % D;
        for (int t = tid / D; t < 256 && c + t < hi; t += SH) {
            if (w[t] == 0.f || !block_of(c + t, half, vhalf, id)) continue;
            const int r = (c + t) & (P - 1);
            if (half) acc += w[t] * bf16_to_f32(vhalf[d * P + r]);
            else
                acc += w[t] * (float)((const int8_t *)a.v)[kv_block_at(a, id, kh) + d * P + r] *
                       a.v_scale[id * a.kv_heads + kh];
        }
        __syncthreads();
        l = l * f + red[0] + red[1] + red[2] + red[3];
        m = mn;
        __syncthreads();
    }
    acc4[tid] = acc;
    __syncthreads();
    if (tid < D) {
        float o = 0.f;
        for (int t = 0; t < SH; ++t) o += acc4[tid + t * D];
        o = l > 0.f || l != l ? o / l : 0.f;
        const int64_t at = ((int64_t)row * a.q_heads + h) * D + tid;
        if (out_f32) ((float *)out)[at] = o;
        else ((__bf16 *)out)[at] = (__bf16)o;
        if (lse && tid == 0) lse[(int64_t)row * a.q_heads + h] = l > 0.f || l != l ? m + __logf(l) : -INFINITY;
    }
}

size_t kv_attention_workspace(const KvArgs &) { return 256; }

template <int D, int BITS>
static hipError_t attend(const KvArgs &a, const uint16_t *q, int64_t q_stride, void *out, int out_f32, float *lse,
                         hipStream_t st)
{
    const int64_t gx = (int64_t)a.n_seq * a.max_rows;
    if (gx > INT32_MAX / 256 || a.q_heads > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_attn_row<D, BITS>), dim3((unsigned)gx, a.q_heads), dim3(256), 0, st, a, q, q_stride, out,
                       out_f32, lse);
    return hipGetLastError();
}

hipError_t launch_kv_attention(const KvArgs &a, const uint16_t *q, int64_t q_stride, void *out, int out_f32, float *lse,
                               void *ws, hipStream_t st)
{
    if (a.head_dim == 64)
        return a.kv_bits == 8 ? attend<64, 8>(a, q, q_stride, out, out_f32, lse, st)
                              : attend<64, 16>(a, q, q_stride, out, out_f32, lse, st);
    return a.kv_bits == 8 ? attend<128, 8>(a, q, q_stride, out, out_f32, lse, st)
                          : attend<128, 16>(a, q, q_stride, out, out_f32, lse, st);
}

}  // namespace moe
