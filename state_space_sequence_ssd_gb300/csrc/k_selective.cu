// k_selective.cu -- the selective scan's forward pass: the hop between chunks, the choice of lanes and chunks, and the
// launches (selective_forward.cuh has the scan itself); and its step for single tokens.
#include "selective.cuh"

namespace ssd {
namespace {

// The states that every chunk starts from: hops[0] = init, hops[k + 1] = exp(A dtsum[k]) hops[k] + (chunk k's own end
// state, which hops[k + 1] holds on entry).  hops and dtsum are written by a launch that may still run when this one
// starts: plain loads behind the wait, from pointers that promise nothing.
__global__ void __launch_bounds__(256) selective_hop_kernel(const float* __restrict__ A, const float* __restrict__ init,
                                                            int channels, int dstate, int nchunks, float* hops,
                                                            const float* dtsum) {
    const int64_t n = (int64_t)channels * dstate, i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int b = blockIdx.y;
    if (i >= n) return;
    const float A2 = A[i] * kLog2e;
    float h = init != nullptr ? init[b * n + i] : 0.f;
    grid_dep_wait();  // the chunks' own states and sums
    float* hp = hops + b * n * nchunks + i;
    const float* dp = dtsum + (int64_t)b * nchunks * channels + i / dstate;
    hp[0] = h;
    // the states and sums of the next chunks are loaded ahead: only the sum waits for the chunk before
    constexpr int AHEAD = 8;
    for (int k = 0; k + 1 < nchunks; k += AHEAD) {
        float own[AHEAD], sum[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (k + u + 1 < nchunks) {
                own[u] = hp[(k + u + 1) * n];
                sum[u] = dp[(int64_t)(k + u) * channels];
            }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (k + u + 1 < nchunks) {
                h = carried(A2 * sum[u], h, own[u]);
                hp[(k + u + 1) * n] = h;
            }
    }
}

}  // namespace

int launch_selective_hop(const SelectiveArgs& a, int nchunks, float* hops, const float* dtsum, cudaStream_t s) {
    launch_begin(kKindSelective, s);
    launch_dependent(selective_hop_kernel, dim3((unsigned)ceil_div64((int64_t)a.channels * a.dstate, 256), a.batch), dim3(256), 0,
                     s, a.A, a.init, a.channels, a.dstate, nchunks, hops, dtsum);
    return launch_end(kKindSelective, s);
}

// Four warps a block, fewer where a group has fewer channels than they cover.
SelectiveShape selective_shape(const SelectiveArgs& a, bool wide) {
    SelectiveShape s = {wide, 1, 128, 0};
    const int entries = wide ? 8 : 4, channels = wide ? 4 : 2, per = a.channels / a.ngroups;
    while (s.lp * entries < a.dstate) s.lp *= 2;
    while (s.threads > 32 && channels * s.threads / 2 / s.lp >= (per < 8 ? 8 : per)) s.threads /= 2;
    s.cc = channels * s.threads / s.lp;
    return s;
}

namespace {

// ------------------------------------------------------------------------------------------------ one token
// A lane holds four state entries of one channel for R rows, and LP lanes share the channel.  Bound by HBM: the state
// is read and written once.  The rows' states are loaded together and A once for them; each of the first R lanes
// forms one row's dt and gate for the others, and ends with that row's output.  An idle row (slot -1) writes zeros
// and leaves every slot alone.  VEC: states, A, B and C are whole vectors of four entries, known when it is compiled.
// 256 rows of 4096 x 16 take 28.7 us, 5.0 TB/s, with 58% of the issue slots used; more bytes in flight do not help: eight rows copied to shared memory ahead 31, two rows or one 33 and 41, a fifth block an SM 36.
template <typename T, int LP, int R, bool VEC>
__global__ void __launch_bounds__(256, 4) selective_step_kernel(SelectiveArgs a, float* __restrict__ state,
                                                             const int* __restrict__ slots, int nslots, T* __restrict__ y,
                                                             int* err, bool some, bool someb) {
    const bool vecs = VEC || some, vecb = VEC || someb;  // states and A; B and C
    const int b0 = blockIdx.y * R, N = a.dstate, q = threadIdx.x % LP;
    const int64_t c = (int64_t)blockIdx.x * (256 / LP) + threadIdx.x / LP;
    const bool mine = c < a.channels;
    const int nvalid = mine ? max(0, min(4, N - 4 * q)) : 0;
    const int g = mine ? (int)(c / (a.channels / a.ngroups)) : 0;
    int slot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) slot[r] = b0 + r < a.batch ? row_slot(slots, b0 + r, nslots, err) : -1;
    Vec<float, 4> h[R];
    Vec<T, 4> Bv[R], Cv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int got = slot[r] >= 0 ? nvalid : 0;
        h[r] = load_vec<float, 4, true>(state + ((int64_t)slot[r] * a.channels + c) * N + 4 * q, got, vecs);
        const int64_t bc = (int64_t)g * N + 4 * q;
        Bv[r] = load_vec<T, 4>(static_cast<const T*>(a.B) + (b0 + r) * a.B_batch + bc, got, vecb);
        Cv[r] = load_vec<T, 4>(static_cast<const T*>(a.C) + (b0 + r) * a.C_batch + bc, got, vecb);
    }
    // lane q: row b0 + q's scalars
    const bool own = mine && q < R && b0 + q < a.batch;
    float xq = 0.f, dq = 0.f, zq = 0.f, Dq = 0.f;
    if (own) {
        xq = to_f32<T>(static_cast<const T*>(a.x)[(b0 + q) * a.x_batch + c]);
        dq = to_f32<T>(static_cast<const T*>(a.dt)[(b0 + q) * a.dt_batch + c]);
        if (a.z != nullptr) zq = to_f32<T>(static_cast<const T*>(a.z)[(b0 + q) * a.z_batch + c]);
        if (a.D != nullptr) Dq = __ldg(a.D + c);
    }
    const float bias = a.dto.bias != nullptr && mine ? __ldg(a.dto.bias + c) : 0.f;
    const Vec<float, 4> A4 = load_vec<float, 4>(a.A + (mine ? c * N + 4 * q : 0), nvalid, vecs);
    const f32x2 log2e = pk(kLog2e, kLog2e), A01 = mul2(A4.pair(0), log2e), A23 = mul2(A4.pair(1), log2e);
    float dv[1] = {dq + bias};
    effective<false>(dv, a.dto);
    dq = dv[0];
    const float dxq = dq * xq;
    float acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float d = __shfl_sync(0xffffffffu, dq, r, LP), dx = __shfl_sync(0xffffffffu, dxq, r, LP);
        const f32x2 dd = pk(d, d), dxx = pk(dx, dx);
        const f32x2 h01 = fma2(exp2_2(mul2(dd, A01)), h[r].pair(0), mul2(dxx, Bv[r].pair(0)));
        const f32x2 h23 = fma2(exp2_2(mul2(dd, A23)), h[r].pair(1), mul2(dxx, Bv[r].pair(1)));
        const f32x2 o[2] = {h01, h23};
        // entries past dstate, whose zeros are NaN once dt x is infinite, are left out of the sum
        if constexpr (VEC) {
            acc[r] = nvalid > 0 ? sum2(fma2(Cv[r].pair(1), h23, mul2(Cv[r].pair(0), h01))) : 0.f;
        } else {
            float p[4], sum = 0.f;
            unpk(mul2(Cv[r].pair(0), h01), p[0], p[1]);
            unpk(mul2(Cv[r].pair(1), h23), p[2], p[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += e < nvalid ? p[e] : 0.f;
            acc[r] = sum;
        }
        if (slot[r] >= 0)
            store_vec<float, 4>(state + ((int64_t)slot[r] * a.channels + c) * N + 4 * q, Vec<float, 4>::of_pairs(o), nvalid, vecs);
    }
    // the rows' sums over the channel's lanes: lane q ends with row `which`
    int which = 0;
    fold_between<R, LP / 2, 1>(acc, q, which);
    // that sum belongs to lane `which` of the channel, which holds the row's x and z; LP / R lanes hold each
    float s = __shfl_sync(0xffffffffu, acc[0], (q % R) * (LP / R), LP);
    if (!own) return;
    int live = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) live |= (r == q && slot[r] >= 0);
    s = fmaf(Dq, xq, s);
    if (a.z != nullptr) s *= zq * sigmoid(zq);
    y[(int64_t)(b0 + q) * a.channels + c] = from_f32<T>(live ? s : 0.f);
}

template <typename T, int LP>
int step_lanes(const SelectiveArgs& a, float* state, const int* slots, int nslots, T* y, int* err, cudaStream_t s) {
    constexpr int R = LP < 4 ? LP : 4;
    const bool vecs = a.dstate % 4 == 0 && aligned_to(state, 16) && aligned_to(a.A, 16), vecb = states_of_four(a, sizeof(T));
    const int tiles = ceil_div(a.channels, 256 / LP);
    launch_begin(kKindSelectiveStep, s);
    auto go = [&](auto kernel, int rows) {
        kernel<<<dim3(tiles, ceil_div(a.batch, rows)), 256, 0, s>>>(a, state, slots, nslots, y, err, vecs, vecb);
    };
    // several rows a thread where the batch fills the SMs all the same (test_layer_sizes_gpu.py has them)
    const bool many = a.batch / R * tiles >= kSms * 4;
    if (vecs && vecb) many ? go(selective_step_kernel<T, LP, R, true>, R) : go(selective_step_kernel<T, LP, 1, true>, 1);
    else many ? go(selective_step_kernel<T, LP, R, false>, R) : go(selective_step_kernel<T, LP, 1, false>, 1);
    return launch_end(kKindSelectiveStep, s);
}

template <typename T>
int step_of(const SelectiveArgs& a, float* state, const int* slots, int nslots, void* y, int* err, cudaStream_t s) {
    T* yt = static_cast<T*>(y);
    switch (selective_lanes(a.dstate)) {
        case 2: return step_lanes<T, 2>(a, state, slots, nslots, yt, err, s);
        case 4: return step_lanes<T, 4>(a, state, slots, nslots, yt, err, s);
        case 8: return step_lanes<T, 8>(a, state, slots, nslots, yt, err, s);
        case 16: return step_lanes<T, 16>(a, state, slots, nslots, yt, err, s);
        case 32: return step_lanes<T, 32>(a, state, slots, nslots, yt, err, s);
        default: return SSD_ERR_UNSUPPORTED;
    }
}

}  // namespace

SelectivePlan selective_plan(const SelectiveArgs& a, int sms) {
    // The lanes and the split into k chunks with the least estimated time.  Clocks of an SM quarter for a token of a chunk,
    // with one, two and three warps on it, measured at bf16 and 16 entries (and for the first run, which all chunks but
    // the last need): wide lanes 640, 740 and 900 (380, 460 and 570), narrow ones, which do a quarter of that work, 250,
    // 290 and 350 (180, 210 and 250) -- so narrow lanes where the SMs would otherwise stay idle.  A split costs two
    // launches and the hop besides, about 5 us and 60 ns a chunk.  What the estimate leaves out: a chunk's states in memory
    // (4 x batch x channels x dstate x 4 bytes), other types and numbers of entries, and that one lane a channel (dstate of 8
    // or less) fits two blocks on an SM, or one in float32, by its shared memory; it says 225 us where 282 are measured at
    // 2 x 4096 x 4096 x 16.
    // Where rows have their own lengths half of the blocks are taken to have work (the others end at once): with lengths
    // spread evenly from nothing to the row 166 us at 8 x 2048 x 2048 x 16 of bfloat16 and 108 at 16 x 512 x 2048 x 16,
    // 192 and 115 with the split for whole rows; with whole rows 285 and 160, 304 and 159; with at least half rows 263 and
    // 144, 252 and 139.
    SelectivePlan best = {true, 1};
    double best_t = -1.0;
    for (int wide = a.dstate <= 16 ? 0 : 1; wide <= 1; ++wide) {
        const SelectiveShape f = selective_shape(a, wide != 0);
        const int64_t blocks = (int64_t)a.batch * a.ngroups * ceil_div(a.channels / a.ngroups, f.cc);
        const int share = a.lengths != nullptr ? 2 : 1;
        const int64_t slots = (int64_t)sms * (3 * 128 / f.threads);
        auto run = [&](int64_t n, double one, double two, double three) {
            const double rest = (double)((n % slots + sms - 1) / sms) * f.threads / 128;  // warps on a quarter in the last wave
            return (double)(n / slots) * three + (rest <= 0 ? 0.0 : rest <= 1 ? one : rest <= 2 ? two : three);
        };
        for (int k = 1; k <= 512 && (k == 1 || a.seqlen / k >= 32); ++k) {
            double t = wide ? run(ceil_div64(blocks * k, share), 640.0, 740.0, 900.0) : run(ceil_div64(blocks * k, share), 250.0, 290.0, 350.0);
            if (k > 1) t += wide ? run(ceil_div64(blocks * (k - 1), share), 380.0, 460.0, 570.0) : run(ceil_div64(blocks * (k - 1), share), 180.0, 210.0, 250.0);
            t *= (double)a.seqlen / k;
            if (k > 1) t += 10000.0 + 120.0 * k;
            if (best_t < 0.0 || t < best_t) {
                best = {wide != 0, k};
                best_t = t;
            }
        }
    }
    return best;
}

size_t selective_workspace(const SelectiveArgs& a, const SelectivePlan& p) {
    return p.chunks > 1 ? (size_t)a.batch * p.chunks * a.channels * (a.dstate + 1) * sizeof(float) : 0;
}

int launch_selective_forward(const SelectiveArgs& a, const SelectivePlan& p, void* y, float* final_state, float* ws,
                             cudaStream_t s) {
    if (a.dtype == SSD_BF16) return selective_forward_bf16(a, p, y, final_state, ws, s);
    if (a.dtype == SSD_F16) return selective_forward_f16(a, p, y, final_state, ws, s);
    return selective_forward_f32(a, p, y, final_state, ws, s);
}

int launch_selective_step(const SelectiveArgs& a, float* state, const int* slots, int nslots, void* y, int* err,
                          cudaStream_t s) {
    if (a.dtype == SSD_BF16) return step_of<__nv_bfloat16>(a, state, slots, nslots, y, err, s);
    if (a.dtype == SSD_F16) return step_of<__half>(a, state, slots, nslots, y, err, s);
    return step_of<float>(a, state, slots, nslots, y, err, s);
}

}  // namespace ssd
