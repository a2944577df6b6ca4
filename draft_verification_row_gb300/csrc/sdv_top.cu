// sdv_top.cu -- the k largest logits of each row in descending order (ties
// by index), their tokens, and the log-sum-exp of all the others at a
// temperature: what a draft model needs of the target's rows to be trained
// on them.
//
// One CTA per row: the maximum, the border of the first k (find_border),
// the kept tokens listed in index order and sorted, then the others' sum
// against the largest of them, so that a tail of 1e-9 of the row's mass
// keeps its digits.
#include "sdv_internal.h"
#include "sdv_rows.cuh"

namespace sdv {
namespace {

template <int DT, int NT>
struct TopSource {
    const Row& row;
    template <class F>
    __device__ __forceinline__ void each(F f) const
    {
        for (int u = threadIdx.x; u < row.n_units; u += NT) {
            float v[Elem<DT>::kPerUnit];
            load_elems<DT>(row, u, v);
#pragma unroll
            for (int e = 0; e < Elem<DT>::kPerUnit; ++e) f(v[e]);
        }
    }
};

template <int NT>
struct TopSmem {
    BlockSmem<NT> bs;
    Hist hist;
    u64 list[SDV_MAX_TOP];  // ~key << 32 | index: ascending is the row's descending order
    float part[NT / 32];
};

// Ascending bitonic sort of n (a power of two) entries in shared memory.
template <int NT>
__device__ void sort_list(u64* list, int n)
{
    for (int size = 2; size <= n; size *= 2) {
        for (int step = size / 2; step > 0; step /= 2) {
            __syncthreads();
            for (int i = threadIdx.x; i < n / 2; i += NT) {
                const int a = 2 * i - (i & (step - 1)), b = a + step;
                const u64 x = list[a], y = list[b];
                if ((x > y) == ((a & size) == 0)) {
                    list[a] = y;
                    list[b] = x;
                }
            }
        }
    }
    __syncthreads();
}

template <int DT, int NT>
__global__ void __launch_bounds__(NT) top_kernel(TopArgs a)
{
    using E = Elem<DT>;
    constexpr int EPU = E::kPerUnit;
    __shared__ TopSmem<NT> sm;
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const Row row = row_at<DT>(a.logits, r, a.stride, a.V);
    float m = -INFINITY;
    for (int u = tid; u < row.n_units; u += NT) m = E::unit_max(load_unit<DT>(row, u), m);
    const float M = block_max_nan<NT>(m, sm.bs);
    const size_t o = (size_t)r * a.k;
    if (!(M > -INFINITY && M < INFINITY)) {
        for (int i = tid; i < a.k; i += NT) {
            a.index[o + i] = -1;
            if (DT == SDV_F32)
                static_cast<float*>(a.values)[o + i] = NAN;
            else
                static_cast<unsigned short*>(a.values)[o + i] = 0x7fc0;
        }
        if (tid == 0) {
            a.rest[r] = NAN;
            if (a.device_status) atomicOr(a.device_status, SDV_REQ_NONFINITE);
        }
        return;
    }
    const TopSource<DT, NT> src{row};
    const uint32_t kmin = lowest_finite_key<DT>();
    Scale none = {};
    const Border b = find_border<DT, NT>(src, false, (u64)a.k, kmin, key_of<DT>(M), none, nullptr, sm.hist, sm.bs);
    const int n = b.found ? a.k : (int)b.above;             // listed tokens
    const int ties = b.found ? a.k - (int)b.above : a.k;    // of the border's key
    // listed in index order, a thread's consecutive units at a time
    const int per = (row.n_units + NT - 1) / NT;
    const int u0 = min(tid * per, row.n_units), u1 = min(u0 + per, row.n_units);
    u64 count = 0;  // above the border's key | of that key << 32
    for (int u = u0; u < u1; ++u) {
        float v[EPU];
        load_elems<DT>(row, u, v);
#pragma unroll
        for (int e = 0; e < EPU; ++e) {
            const uint32_t k = key_of<DT>(v[e]);
            count += k > b.key ? 1ull : k == b.key ? 1ull << 32 : 0ull;
        }
    }
    u64 total;
    u64 at = block_scan<NT>(count, total, sm.bs);
    float next = -INFINITY;  // the largest of the others
    for (int u = u0; u < u1; ++u) {
        float v[EPU];
        load_elems<DT>(row, u, v);
#pragma unroll
        for (int e = 0; e < EPU; ++e) {
            const uint32_t k = key_of<DT>(v[e]);
            const int before = (int)(uint32_t)at, tied = (int)(at >> 32);
            if (k > b.key || (k == b.key && tied < ties))
                sm.list[before + min(tied, ties)] = (u64)~k << 32 | (uint32_t)(u * EPU + e - row.off);
            else
                next = fmaxf(next, v[e]);
            at += k > b.key ? 1ull : k == b.key ? 1ull << 32 : 0ull;
        }
    }
    next = block_max_nan<NT>(next, sm.bs);
    int n2 = 1;
    while (n2 < n) n2 *= 2;
    for (int i = n + tid; i < n2; i += NT) sm.list[i] = ~0ull;
    __syncthreads();
    // the last kept index of the border's key, in index order
    int last = -1;
    for (int i = tid; i < n; i += NT)
        if (~(uint32_t)(sm.list[i] >> 32) == b.key) last = max(last, (int)(uint32_t)sm.list[i]);
    last = __reduce_max_sync(0xffffffffu, last);
    __syncthreads();
    if (lane == 0) sm.part[w] = __int_as_float(last);
    __syncthreads();
    for (int i = 0; i < NT / 32; ++i) last = max(last, __float_as_int(sm.part[i]));
    sort_list<NT>(sm.list, n2);
    for (int i = tid; i < a.k; i += NT) {
        const float x = i < n ? key_value<DT>(~(uint32_t)(sm.list[i] >> 32)) : -INFINITY;
        a.index[o + i] = i < n ? (int)(uint32_t)sm.list[i] : -1;
        if (DT == SDV_F32)
            static_cast<float*>(a.values)[o + i] = x;
        else
            static_cast<unsigned short*>(a.values)[o + i] = (unsigned short)(__float_as_uint(x) >> 16);
    }
    float z = 0.f;
    if (next > -INFINITY) {
        const float c = (float)a.c;
        for (int u = tid; u < row.n_units; u += NT) {
            float v[EPU];
            load_elems<DT>(row, u, v);
#pragma unroll
            for (int e = 0; e < EPU; ++e) {
                const uint32_t k = key_of<DT>(v[e]);
                const bool listed = k > b.key || (k == b.key && u * EPU + e - row.off <= last);
                z += listed ? 0.f : ex2((v[e] - next) * c);
            }
        }
    }
    z = warp_sum(z);
    __syncthreads();
    if (lane == 0) sm.part[w] = z;
    __syncthreads();
    if (tid == 0) {
        z = 0.f;
        for (int i = 0; i < NT / 32; ++i) z += sm.part[i];
        a.rest[r] = next > -INFINITY ? (float)((double)next * a.inv_T + (double)logf(z)) : -INFINITY;
    }
}

}  // namespace

cudaError_t launch_top(const TopArgs& a, cudaStream_t st)
{
    if (a.dtype == SDV_F32)
        top_kernel<SDV_F32, 512><<<a.n_rows, 512, 0, st>>>(a);
    else
        top_kernel<SDV_BF16, 512><<<a.n_rows, 512, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace sdv
