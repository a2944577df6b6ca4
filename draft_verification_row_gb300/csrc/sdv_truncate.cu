// sdv_truncate.cu -- truncated sampling and truncated rows: the first
// tokens of a row's descending order that top-k, top-p and min-p all keep,
// drawn from (the draft tokens of speculative decoding as servers draw
// them) or written as a row of logits that the verification rules read.
//
// With w_i = exp((x_i - max) / T) and the order by value, then by index:
//   n_k = top_k (all if 0), Z_k the sum of the first n_k weights;
//   n_p = least n whose first n weights sum to top_p Z_k or more;
//   n_m = number of tokens with (x_i - max) / T >= ln(min_p);
// the first max(1, min(n_k, n_p, n_m)) tokens are kept.  All three keep a
// prefix of one order, so the kept set is a border: a key, and the index of
// the last token of that key that is kept.
//
// One CTA per row.  The row is read from HBM once, for its maximum; what
// follows reads it from L2.  All masses are fixed-point integers
// (weight_of), so every run gives the same tokens.
#include "sdv_internal.h"
#include "sdv_rows.cuh"

namespace sdv {
namespace {

constexpr int kSegU = 256;                                       // units per segment: a warp's step of 8 per lane
constexpr int kMaxSeg = (SDV_MAX_V / 4 + 1 + kSegU - 1) / kSegU;  // segments of the longest row

template <int NT>
struct TruncSmem {
    BlockSmem<NT> bs;
    Hist hist;
    u64 table[64];
    u64 seg[kMaxSeg];  // per segment: tied tokens, then kept mass
    int last;          // index of the last kept token of the border's key
};

// The elements of a row, by threads: unit tid, tid + NT, ...
template <int DT, int NT>
struct RowSource {
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

// The kept set: tokens with a key above `key`, and those of that key up to
// index `last`.
struct Kept {
    uint32_t key;
    int last;
};

template <int DT>
__device__ __forceinline__ bool is_kept(float x, int i, const Kept& c)
{
    const uint32_t k = key_of<DT>(x);
    return k > c.key || (k == c.key && i <= c.last);
}

// Per segment, the sum of f(x, index) over its elements, into seg[].
template <int DT, int NT, class F>
__device__ void segment_sums(const Row& row, u64* seg, F f)
{
    constexpr int EPU = Elem<DT>::kPerUnit;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int n_seg = (row.n_units + kSegU - 1) / kSegU;
    for (int s = w; s < n_seg; s += NT / 32) {
        u64 sum = 0;
        for (int u = s * kSegU + lane; u < min((s + 1) * kSegU, row.n_units); u += 32) {
            float v[EPU];
            load_elems<DT>(row, u, v);
#pragma unroll
            for (int e = 0; e < EPU; ++e) sum += f(v[e], u * EPU + e - row.off);
        }
        sum = warp_sum_u64(sum);
        if (lane == 0) seg[s] = sum;
    }
}

// The first index, in index order, at which the running sum of f exceeds
// thr (one warp; seg[] holds the segments' sums): -1 if none does.
template <int DT, class F>
__device__ int crossing(const Row& row, const u64* seg, u64 thr, F f)
{
    constexpr int EPU = Elem<DT>::kPerUnit;
    const int lane = threadIdx.x & 31;
    const int n_seg = (row.n_units + kSegU - 1) / kSegU;
    u64 run = 0;
    int s = -1;
    for (int s0 = 0; s0 < n_seg; s0 += 32) {
        const u64 v = s0 + lane < n_seg ? seg[s0 + lane] : 0;
        const u64 incl = run + warp_scan_u64(v, lane);
        const unsigned over = __ballot_sync(0xffffffffu, incl > thr);
        if (over) {
            const int l = __ffs(over) - 1;
            s = s0 + l;
            run = __shfl_sync(0xffffffffu, incl - v, l);
            break;
        }
        run = __shfl_sync(0xffffffffu, incl, 31);
    }
    if (s < 0) return -1;
    for (int u0 = s * kSegU; u0 < min((s + 1) * kSegU, row.n_units); u0 += 32) {
        const int u = u0 + lane;
        u64 g[EPU], sum = 0;
#pragma unroll
        for (int e = 0; e < EPU; ++e) g[e] = 0;
        if (u < row.n_units) {
            float v[EPU];
            load_elems<DT>(row, u, v);
#pragma unroll
            for (int e = 0; e < EPU; ++e) {
                g[e] = f(v[e], u * EPU + e - row.off);
                sum += g[e];
            }
        }
        const u64 incl = run + warp_scan_u64(sum, lane);
        const unsigned over = __ballot_sync(0xffffffffu, incl > thr);
        if (over) {
            const int l = __ffs(over) - 1;
            int pick = -1;
            u64 acc = incl - sum;
#pragma unroll
            for (int e = 0; e < EPU; ++e) {
                acc += g[e];
                if (pick < 0 && acc > thr) pick = u * EPU + e - row.off;
            }
            return __shfl_sync(0xffffffffu, pick, l);
        }
        run = __shfl_sync(0xffffffffu, incl, 31);
    }
    return -1;
}

// A row's settings.
struct Settings {
    float T;
    int k;
    float p, m;
    bool ok;
};

__device__ __forceinline__ Settings settings_of(const TruncArgs& a, int r)
{
    Settings s;
    s.T = a.row_temperature ? a.row_temperature[r] : a.temperature;
    s.k = a.row_top_k ? a.row_top_k[r] : a.top_k;
    s.p = a.row_top_p ? a.row_top_p[r] : a.top_p;
    s.m = a.row_min_p ? a.row_min_p[r] : a.min_p;
    // T >= 0 with a finite log2(e) / T
    s.ok = s.T == 0.f || (s.T >= 4.3e-39f && s.T < INFINITY);
    s.ok = s.ok && s.k >= 0 && s.p > 0.f && s.p <= 1.f && s.m >= 0.f && s.m <= 1.f;
    return s;
}

// The kept set of a row whose maximum is finite (all threads).
template <int DT, int NT>
__device__ Kept find_kept(const Row& row, const Settings& st, const Scale& sc, TruncSmem<NT>& sm)
{
    const uint32_t kmax = key_of<DT>(sc.M), kmin = lowest_finite_key<DT>();
    const RowSource<DT, NT> src{row};
    uint32_t key = kmin;
    u64 ties = ~0ull;  // tokens of that key that are kept
    if (st.T == 0.f) {
        key = kmax;
        ties = 1;
    } else {
        if (st.k > 0 && st.k < row.V) {
            const Border b = find_border<DT, NT>(src, false, (u64)st.k, kmin, kmax, sc, sm.table, sm.hist, sm.bs);
            if (b.found) {
                key = b.key;
                ties = (u64)st.k - b.above;
            }
        }
        if (st.p < 1.f) {
            // the mass of the first n_k tokens, and the border of its share
            // p; tokens of the k-th key enter by their number
            const bool limited = ties != ~0ull;
            u64 mass = 0;
            src.each([&](float x) {
                const uint32_t k = key_of<DT>(x);
                if (k > key || (k == key && !limited)) mass += weight_of(x, sc, sm.table);
            });
            mass = block_sum<NT>(mass, sm.bs);
            const u64 w_tie = limited ? weight_of(key_value<DT>(key), sc, sm.table) : 0;
            const u64 Z = mass + (limited ? ties * w_tie : 0);
            u64 need = (u64)ceil((double)st.p * (double)Z);
            if (need < 1) need = 1;
            if (mass >= need) {
                const Border b = find_border<DT, NT>(src, true, need, limited ? key + 1 : key, kmax, sc, sm.table,
                                                     sm.hist, sm.bs);
                const u64 w = weight_of(key_value<DT>(b.key), sc, sm.table);
                key = b.key;
                ties = (need - b.above + w - 1) / w;
            } else if (w_tie > 0) {  // among the tokens of the k-th key
                const u64 t = (need - mass + w_tie - 1) / w_tie;
                if (t < ties) ties = t;
            }
        }
        if (st.m > 0.f) {
            const float x = __double2float_ru((double)sc.M + (double)st.T * log((double)st.m));
            uint32_t k = key_of<DT>(x);
            if (key_value<DT>(k) < x) ++k;  // the next bf16 value up
            if (k > key) {
                key = k;
                ties = ~0ull;
            }
        }
    }
    // the index of the last kept token of the border's key
    Kept c;
    c.key = key;
    c.last = 0x7fffffff;
    if (ties != ~0ull) {
        segment_sums<DT, NT>(row, sm.seg, [&](float x, int) { return (u64)(key_of<DT>(x) == key ? 1 : 0); });
        __syncthreads();
        if (threadIdx.x < 32) {
            const int i = crossing<DT>(row, sm.seg, ties - 1,
                                       [&](float x, int) { return (u64)(key_of<DT>(x) == key ? 1 : 0); });
            if (threadIdx.x == 0) sm.last = i < 0 ? 0x7fffffff : i;
        }
        __syncthreads();
        c.last = sm.last;
    }
    return c;
}

// The row with what is not kept at -inf (bad: as it is).  Aligned alike,
// input and output move as 16-byte units; else element by element.
template <int DT, int NT>
__device__ void write_row(const Row& row, void* out, const Kept& c, bool bad)
{
    constexpr int EPU = Elem<DT>::kPerUnit;
    const Row o = row_at<DT>(out, 0, 0, row.V);
    const bool alike = o.off == row.off;
    for (int u = threadIdx.x; u < row.n_units; u += NT) {
        uint4 raw = load_unit<DT>(row, u);
        float v[EPU];
        Elem<DT>::unpack(raw, v);
        uint32_t keep = 0;
#pragma unroll
        for (int e = 0; e < EPU; ++e) keep |= (bad || is_kept<DT>(v[e], u * EPU + e - row.off, c) ? 1u : 0u) << e;
        uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (DT == SDV_F32) {
                if (!(keep >> i & 1)) w[i] = 0xff800000u;
            } else {
                if (!(keep >> (2 * i) & 1)) w[i] = (w[i] & 0xffff0000u) | 0xff80u;
                if (!(keep >> (2 * i + 1) & 1)) w[i] = (w[i] & 0xffffu) | 0xff800000u;
            }
        }
        if (alike && whole_unit<DT>(row, u)) {
            reinterpret_cast<uint4*>(o.p)[u] = make_uint4(w[0], w[1], w[2], w[3]);
            continue;
        }
#pragma unroll
        for (int e = 0; e < EPU; ++e) {
            const int x = u * EPU + e - row.off;
            if (x < 0 || x >= row.V) continue;
            if (DT == SDV_F32)
                static_cast<uint32_t*>(out)[x] = w[e % 4];
            else
                static_cast<unsigned short*>(out)[x] = (unsigned short)(w[e / 2 % 4] >> (e & 1) * 16);
        }
    }
}

template <int DT, int NT>
__global__ void __launch_bounds__(NT) truncate_kernel(TruncArgs a)
{
    using E = Elem<DT>;
    __shared__ TruncSmem<NT> sm;
    const int r = blockIdx.x;
    const int tid = threadIdx.x;
    for (int i = tid; i < 64; i += NT) sm.table[i] = kExp2Table[i];
    const Row row = row_at<DT>(a.logits, r, a.stride, a.V);
    const Settings st = settings_of(a, r);
    float m = -INFINITY;
    for (int u = tid; u < row.n_units; u += NT) m = E::unit_max(load_unit<DT>(row, u), m);
    Scale sc;
    sc.M = block_max_nan<NT>(m, sm.bs);
    const bool finite = sc.M > -INFINITY && sc.M < INFINITY;
    int* const tokens = a.tokens ? a.tokens + (size_t)r * a.n_samples : nullptr;
    char* const out = a.out ? static_cast<char*>(a.out) + (size_t)r * (size_t)a.out_stride * E::kBytes : nullptr;
    Kept c = {0u, 0};
    if (!finite || !st.ok) {
        if (tokens)
            for (int s = tid; s < a.n_samples; s += NT) tokens[s] = -1;
        if (out) write_row<DT, NT>(row, out, c, true);
        if (tid == 0 && a.device_status)
            atomicOr(a.device_status, (finite ? 0 : SDV_REQ_NONFINITE) | (st.ok ? 0 : SDV_REQ_BAD_SETTING));
        return;
    }
    const double cc = st.T > 0.f ? 1.4426950408889634 / (double)st.T : 0.0;
    sc.ch = (float)cc;
    sc.cl = (float)(cc - (double)sc.ch);
    c = find_kept<DT, NT>(row, st, sc, sm);
    if (out) write_row<DT, NT>(row, out, c, false);
    if (!tokens) return;
    const auto mass = [&](float x, int i) {
        return is_kept<DT>(x, i, c) ? (st.T > 0.f ? weight_of(x, sc, sm.table) : 1ull) : 0ull;
    };
    __syncthreads();
    segment_sums<DT, NT>(row, sm.seg, mass);
    __syncthreads();
    u64 S = 0;
    for (int i = tid & 31; i < (row.n_units + kSegU - 1) / kSegU; i += 32) S += sm.seg[i];
    S = warp_sum_u64(S);
    for (int s = tid >> 5; s < a.n_samples; s += NT / 32) {
        // u S < S for u < 1; a uniform outside [0, 1) gives the first or
        // the last token
        const double u = a.u ? (double)a.u[(size_t)r * a.n_samples + s] : 0.0;
        u64 thr = u > 0.0 ? (u64)(fmin(u, 1.0) * (double)S) : 0;
        if (thr >= S) thr = S - 1;
        const int i = crossing<DT>(row, sm.seg, thr, mass);
        if ((tid & 31) == 0) tokens[s] = i;
    }
}

template <int DT>
cudaError_t launch(const TruncArgs& a, cudaStream_t st)
{
    truncate_kernel<DT, 512><<<a.n_rows, 512, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_truncate(const TruncArgs& a, cudaStream_t st)
{
    return a.dtype == SDV_F32 ? launch<SDV_F32>(a, st) : launch<SDV_BF16>(a, st);
}

}  // namespace sdv
