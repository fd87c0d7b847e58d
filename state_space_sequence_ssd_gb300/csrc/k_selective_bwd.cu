// k_selective_bwd.cu -- the gradients of the selective scan: the cut into blocks, the hops between them and the sums of
// their parts (selective_backward.cuh has the work on the blocks, and the mathematics).
#include "selective.cuh"

namespace ssd {
namespace {

// hops[k]: the state that block k starts from; mus[k]: the gradient that reaches the state after block k from later
// tokens; dinit.  The four workspaces are written by a launch that may still run when this one starts: plain loads behind
// the wait, from pointers that promise nothing.
__global__ void __launch_bounds__(256) selective_hops_kernel(const float* __restrict__ A, const float* __restrict__ init,
                                                             const float* __restrict__ dfinal, int channels, int dstate,
                                                             int nblocks, float* hops, float* mus, const float* nu0,
                                                             const float* dtsum, float* __restrict__ dinit) {
    const int64_t n = (int64_t)channels * dstate, i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int b = blockIdx.y;
    if (i >= n) return;
    const float A2 = A[i] * kLog2e;
    const float* dp = dtsum + (int64_t)b * nblocks * channels + i / dstate;
    const bool back = blockIdx.z != 0;
    float* at = (back ? mus : hops) + b * n * nblocks + (back ? (nblocks - 1) * n : 0) + i;
    const int64_t step = back ? -n : n, dstep = back ? -channels : channels;
    if (back) dp += (int64_t)(nblocks - 1) * channels;
    const float* start = back ? dfinal : init;
    float s = start != nullptr ? start[b * n + i] : 0.f;
    grid_dep_wait();  // the blocks' own terms
    // the terms of the next blocks are loaded ahead: only the sum waits for the block before
    constexpr int AHEAD = 8;
    *at = s;
    for (int k = 0; k + 1 < nblocks; k += AHEAD) {
        float term[AHEAD], sum[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (k + u + 1 < nblocks) {
                term[u] = at[(u + 1) * step];
                sum[u] = dp[u * dstep];
            }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (k + u + 1 < nblocks) {
                s = carried(A2 * sum[u], s, term[u]);
                at[(u + 1) * step] = s;
            }
        at += AHEAD * step;
        dp += AHEAD * dstep;
    }
    if (back && dinit != nullptr)
        dinit[b * n + i] = carried(A2 * dtsum[(int64_t)b * nblocks * channels + i / dstate], s, nu0[b * n + i]);
}

// What the blocks' parts are added to, in one launch: thread blocks of three kinds after one another.  dA and then dD and
// ddt_bias are sums over rows, eight strided ones and then those eight; dB and dC sums over the tiles of channels.
struct Sums {
    const float *dA_parts, *chan, *dbc;
    float *dA, *dD, *dbias, *dB, *dC;
    int64_t n, tokens;  // channels x entries; tokens x groups
    int rows, channels, tiles, dstate;
    int a_blocks, d_blocks;
};
__global__ void __launch_bounds__(256) selective_sums_kernel(Sums u) {
    __shared__ float part[8][33];
    int block = blockIdx.x;
    grid_dep_wait();
    if (block >= u.a_blocks + u.d_blocks) {
        const int64_t i = (int64_t)(block - u.a_blocks - u.d_blocks) * 256 + threadIdx.x, n = u.tokens * 2 * u.dstate;
        if (i >= n) return;
        float s = 0.f;
#pragma unroll 8
        for (int t = 0; t < u.tiles; ++t) s += u.dbc[t * n + i];
        const int64_t row = i / (2 * u.dstate);
        const int e = (int)(i % (2 * u.dstate));
        if (e < u.dstate) u.dB[row * u.dstate + e] = s;
        else u.dC[row * u.dstate + e - u.dstate] = s;
        return;
    }
    const bool channels = block >= u.a_blocks;
    if (channels) block -= u.a_blocks;
    const float* in = channels ? u.chan : u.dA_parts;
    const int64_t n = channels ? 2 * u.channels : u.n;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = (int64_t)block * 32 + lane;
    float s = 0.f;
    if (i < n) {
#pragma unroll 8
        for (int r = warp; r < u.rows; r += 8) s += in[r * n + i];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || i >= n) return;
    s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += part[q][lane];
    if (!channels) u.dA[i] = s;
    else if (i < u.channels && u.dD != nullptr) u.dD[i] = s;
    else if (i >= u.channels && u.dbias != nullptr) u.dbias[i - u.channels] = s;
}

}  // namespace

int launch_selective_hops(const SelectiveArgs& a, const SelectiveGrads& g, const SelectiveParts& p, float* hops, float* mus,
                          const float* nu0, const float* dtsum, cudaStream_t s) {
    launch_begin(kKindSelectiveBwd, s);
    launch_dependent(selective_hops_kernel, dim3((unsigned)ceil_div64((int64_t)a.channels * a.dstate, 256), a.batch, 2),
                     dim3(256), 0, s, a.A, a.init, g.dfinal, a.channels, a.dstate, p.nblocks, hops, mus, nu0, dtsum, g.dinit);
    return launch_end(kKindSelectiveBwd, s);
}

int launch_selective_sums(const SelectiveArgs& a, const SelectiveGrads& g, const SelectiveParts& p, const float* dA_parts,
                          const float* chan, const float* dbc, cudaStream_t s) {
    const int64_t n = (int64_t)a.channels * a.dstate;
    Sums u = {dA_parts, chan, dbc, g.dA, g.dD, g.ddt_bias, g.dB, g.dC, n, (int64_t)a.batch * a.seqlen * a.ngroups,
              a.batch * p.nblocks, a.channels, p.tiles, a.dstate, (int)ceil_div64(n, 32), 0};
    if (g.dD != nullptr || g.ddt_bias != nullptr) u.d_blocks = ceil_div(2 * a.channels, 32);
    const int64_t blocks = u.a_blocks + u.d_blocks + ceil_div64(u.tokens * 2 * a.dstate, 256);
    if (blocks > 2147483647) return SSD_ERR_UNSUPPORTED;
    launch_begin(kKindSelectiveBwd, s);
    launch_dependent(selective_sums_kernel, dim3((unsigned)blocks), dim3(256), 0, s, u);
    return launch_end(kKindSelectiveBwd, s);
}

// Threads of a block: four warps (two where two lanes share a channel: shared memory), fewer where a group has fewer
// channels than they cover.
int selective_block_threads(const SelectiveArgs& a) {
    const int lp = selective_lanes(a.dstate), per = a.channels / a.ngroups;
    int threads = lp == 2 ? 64 : 128;
    while (threads > 32 && 4 * threads / 2 / lp >= per) threads /= 2;
    return threads;
}

// Blocks of 32 tokens, or of 16 where those of 32 would leave an SM quarter without a warp: half a block's time for twice
// the hops, sums and checkpoints.  With 32 and with 16 tokens at 16 entries of bfloat16: 34 and 21 us at 2 x 128 x 512, 35
// and 28 at 512 x 1024, 47 and 50 at 4 x 64 x 4096, 139 and 150 at 2 x 1024 x 2048.  Rows that fit 32 tokens need no hop.
// (test_layer_sizes_gpu.py has the blocks of 32 for every number of lanes.)
constexpr int kFewWarps = kSms * 4;
static_assert(kFewWarps * 2 <= kMaxGrid, "blocks of 16 tokens fit the grid");
SelectiveParts selective_parts(const SelectiveArgs& a) {
    SelectiveParts p;
    const int threads = selective_block_threads(a), lp = selective_lanes(a.dstate);
    p.tiles = ceil_div(a.channels / a.ngroups, 4 * threads / lp);
    const int64_t warps = (int64_t)a.batch * a.ngroups * p.tiles * ceil_div(a.seqlen, 32) * (threads / 32);
    p.tokens = lp <= 16 && warps <= kFewWarps && (a.seqlen <= 16 || a.seqlen > 32) ? 16 : 32;
    p.nblocks = ceil_div(a.seqlen, p.tokens);
    const size_t n = (size_t)a.channels * a.dstate, rows = (size_t)a.batch * p.nblocks;
    auto whole = [](size_t floats) { return (floats + 3) & ~(size_t)3; };  // every part starts on 16 bytes
    p.hops = whole(rows * n);
    p.nu0 = whole(a.batch * n);
    p.dtsum = whole(rows * a.channels);
    p.chan = whole(2 * rows * a.channels);
    p.dbc = (size_t)p.tiles * a.batch * a.seqlen * a.ngroups * 2 * a.dstate;
    return p;
}

size_t selective_backward_workspace(const SelectiveArgs& a) { return selective_parts(a).total() * sizeof(float); }

int launch_selective_backward(const SelectiveArgs& a, const SelectiveGrads& g, float* ws, cudaStream_t s) {
    if (a.dtype == SSD_BF16) return selective_backward_bf16(a, g, ws, s);
    if (a.dtype == SSD_F16) return selective_backward_f16(a, g, ws, s);
    return selective_backward_f32(a, g, ws, s);
}

}  // namespace ssd
