// k_rotary.cu -- rotary positions: pairs of a head's entries turned by an angle that grows with the token's position.
//
//   (a, b) -> scale (a cos - b sin, a sin + b cos),   angle = position * frequency[pair]
//
// The table holds each pair's frequency as the part of a turn that one position adds, in units of 2^-64: the product with a position,
// taken modulo 2^64, is the angle with its whole turns gone, exactly, at any position and without a float64 operation.  Its
// upper 32 bits are the angle to 2^-32 of a turn.
// Bound by HBM: every entry is read and written once.  A thread turns the same pairs of up to four heads, so that they share the
// sine and cosine; the two tensors' heads (a scan's B and C) go side by side in one launch.  262144 tokens of 2 x 8 x 256 of bfloat16
// take 613 us: 7.0 TB/s, the rate of a plain copy.
#include "ops.cuh"

namespace ssd {
namespace {

constexpr int kRotaryThreads = 256;

// cos and sin of `turns`, the signed fraction of a turn in units of 2^-32.
// float32 tensors: the next whole quarter turn is taken out of the integer, and what is left, t half turns within a quarter, rounded to
// float32: to 2^-24 of itself, where a turn rounded whole would move a sine near half a turn by up to 1.6 2^-24.  sin(pi t) / t and
// (cos(pi t) - 1) / t^2 are polynomials in t^2, interpolated at the Chebyshev nodes of [0, 1/16] with four coefficients (largest errors 0.04
// and 0.003 2^-24 of the sine and the cosine), pi in two parts; with t's rounding both are within 1.9 2^-24 of themselves (6 million samples).
// The other types take the special function unit's, whose absolute error on [-pi, pi] of 2^-20 is far below half a step of their
// type (2^-11 and more).
template <typename T>
__device__ __forceinline__ void cos_sin(int turns, float& c, float& s) {
    if constexpr (sizeof(T) == 4) {
        const unsigned quarter = ((unsigned)turns + 0x20000000u) >> 30;
        const float t = (float)(int)((unsigned)turns - (quarter << 30)) * 0x1p-31f, z = t * t;
        float p = fmaf(z, -0.5890751f, 2.549767f), q = fmaf(z, 0.23212542f, -1.3351378f);
        p = fmaf(z, fmaf(z, p, -5.167708f), -9.71061e-8f);  // from pi's rest on
        q = fmaf(z, fmaf(z, q, 4.0587106f), -4.934802f);
        const float s0 = fmaf(t, 3.1415927f, t * p), c0 = fmaf(z, q, 1.f);
        c = __uint_as_float(__float_as_uint(quarter & 1 ? s0 : c0) ^ (((quarter + 1) & 2) << 30));
        s = __uint_as_float(__float_as_uint(quarter & 1 ? c0 : s0) ^ ((quarter & 2) << 30));
    } else {
        const float v = (float)turns * (6.283185307179586f * 0x1p-32f);
        asm("sin.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(v));
        asm("cos.approx.ftz.f32 %0, %1;" : "=f"(c) : "f"(v));
    }
}

// V: entries of a vector.  HALF: pairs (k, k + turned / 2), a thread holding V pairs of a head in two vectors; else (2 k, 2 k + 1), V / 2
// pairs in one.  H: heads a thread.  `chunks` vectors (or pairs of vectors) a head, `blocks` groups of H heads.
template <typename T, int V, bool HALF, int H>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(RotaryArgs g, int chunks, int blocks, int tokens, bool vec) {
    constexpr int NP = HALF ? V : V / 2;
    const int per = chunks * blocks, b = blockIdx.y;
    const int share = per < kRotaryThreads ? per : kRotaryThreads;  // threads of a token
    const int t = blockIdx.x * tokens + threadIdx.x / share;
    if ((int)threadIdx.x >= tokens * share || t >= g.seqlen) return;
    const bool live = t < row_length(g.lengths, b, g.seqlen);
    int64_t position = t;
    if (g.positions != nullptr) position = g.each ? g.positions[(int64_t)b * g.seqlen + t] : position + g.positions[b];
    const int pairs = g.turned / 2, turning = HALF ? ceil_div(pairs, V) : chunks;
    for (int unit = threadIdx.x % share; unit < per; unit += share) {
        const int chunk = unit % chunks, head0 = unit / chunks * H;
        const bool turn = chunk < turning;
        const int c0 = turn ? chunk * V : g.turned + (chunk - turning) * V, c1 = c0 + pairs;
        const int left0 = (HALF && turn ? pairs : g.dim) - c0, left1 = HALF && turn ? pairs - chunk * V : 0;
        Vec<T, V> r0[H], r1[H];
        const T* from[H];
        T* to[H];
#pragma unroll
        for (int k = 0; k < H; ++k) {
            const int head = head0 + k, second = head >= g.heads[0], h = head - (second ? g.heads[0] : 0);
            const bool in = head < g.heads[0] + g.heads[1];
            from[k] = in ? static_cast<const T*>(g.in[second]) + b * g.batch_stride[second] + t * g.token_stride[second] + (int64_t)h * g.dim : nullptr;
            to[k] = in ? static_cast<T*>(g.out[second]) + (((int64_t)b * g.seqlen + t) * g.heads[second] + h) * g.dim : nullptr;
            const bool read = in && live;
            r0[k] = load_vec<T, V>(read ? from[k] + c0 : nullptr, read ? left0 : 0, vec);
            if (HALF) r1[k] = load_vec<T, V>(read ? from[k] + c1 : nullptr, read ? left1 : 0, vec);
        }
        float cs[NP], sn[NP];
        if (turn) {
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int k = (HALF ? chunk * V : chunk * V / 2) + p;
                cs[p] = sn[p] = 0.f;
                if (k < pairs) {
                    cos_sin<T>((int)(((unsigned long long)position * __ldg(g.table + k)) >> 32), cs[p], sn[p]);
                    cs[p] *= g.scale;
                    sn[p] *= g.inverse ? -g.scale : g.scale;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < H; ++k) {
            if (to[k] == nullptr) break;
            if (turn) {
                float o0[V], o1[V];
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const float x = HALF ? r0[k].get(p) : r0[k].get(2 * p % V), y = HALF ? r1[k].get(p) : r0[k].get((2 * p + 1) % V);
                    const bool in = HALF || chunk * V / 2 + p < pairs;  // a vector may hold entries that are copied
                    const float first = in ? fmaf(x, cs[p], -y * sn[p]) : x, other = in ? fmaf(x, sn[p], y * cs[p]) : y;
                    if (HALF) {
                        o0[p] = first;
                        o1[p] = other;
                    } else {
                        o0[2 * p % V] = first;
                        o0[(2 * p + 1) % V] = other;
                    }
                }
                r0[k] = Vec<T, V>::of(o0);
                if (HALF) r1[k] = Vec<T, V>::of(o1);
            }
            store_vec<T, V>(to[k] + c0, r0[k], left0, vec);
            if (HALF) store_vec<T, V>(to[k] + c1, r1[k], left1, vec);
        }
    }
}

template <typename T, int V, bool HALF>
int rotary_of(const RotaryArgs& g, bool vec, cudaStream_t s) {
    const int pairs = g.turned / 2, heads = g.heads[0] + g.heads[1];
    const int chunks = HALF ? ceil_div(pairs, V) + ceil_div(g.dim - g.turned, V) : ceil_div(g.dim, V);
    // Four heads a thread where that leaves every SM 384 threads (B and C of 8 x 128, one and four heads a thread: 1024 tokens of bfloat16
    // 4.05 and 4.25 us, 2048 6.0 and 5.2, 4096 9.0 and 7.9; 2048 of float32 10.4 and 7.5).
    const bool many = (int64_t)g.batch * g.seqlen * chunks * ceil_div(heads, 4) >= (int64_t)kSms * 384;
    const int blocks = ceil_div(heads, many ? 4 : 1);
    const int64_t per = (int64_t)chunks * blocks;
    if (per > 2147483647) return SSD_ERR_UNSUPPORTED;
    const int tokens = per >= kRotaryThreads ? 1 : kRotaryThreads / (int)per;
    const dim3 grid(ceil_div(g.seqlen, tokens), g.batch);
    launch_begin(kKindRotary, s);
    if (many) rotary_kernel<T, V, HALF, 4><<<grid, kRotaryThreads, 0, s>>>(g, chunks, blocks, tokens, vec);
    else rotary_kernel<T, V, HALF, 1><<<grid, kRotaryThreads, 0, s>>>(g, chunks, blocks, tokens, vec);
    return launch_end(kKindRotary, s);
}

template <typename T, int V>
int rotary_vectors(const RotaryArgs& g, cudaStream_t s) {
    return g.interleaved ? rotary_of<T, V, false>(g, true, s) : rotary_of<T, V, true>(g, true, s);
}

// The widest vectors of which rows, heads and (half layout) halves are whole and aligned; else an element at a time, two pairs a thread
// (B and C of 8 x 2560 tokens of float16: 8 x 48 in vectors of eight 14 us, 8 x 44 interleaved of four 19, half layout of two 23; 8 x 46
// of odd rows an element at a time, half layout: one pair a thread 41, two 32, four 46; interleaved one pair 37, two 31, and one as
// a vector where rows allow it 35).
template <typename T>
int rotary_type(const RotaryArgs& g, cudaStream_t s) {
    constexpr int FULL = 16 / sizeof(T);
    auto fits = [&](int V) {
        bool whole = g.dim % V == 0 && (g.interleaved || g.turned / 2 % V == 0);
        for (int k = 0; k < 2; ++k)
            if (g.heads[k] > 0)
                whole = whole && g.batch_stride[k] % V == 0 && g.token_stride[k] % V == 0 && aligned_to(g.in[k], V * sizeof(T)) && aligned_to(g.out[k], V * sizeof(T));
        return whole;
    };
    if (fits(FULL)) return rotary_vectors<T, FULL>(g, s);
    if (FULL > 4 && fits(4)) return rotary_vectors<T, 4>(g, s);
    if (!g.interleaved && fits(2)) return rotary_of<T, 2, true>(g, true, s);
    return g.interleaved ? rotary_of<T, 4, false>(g, false, s) : rotary_of<T, 2, true>(g, false, s);
}

}  // namespace

int launch_rotary(const RotaryArgs& g, cudaStream_t s) {
    if (g.dtype == SSD_BF16) return rotary_type<__nv_bfloat16>(g, s);
    if (g.dtype == SSD_F16) return rotary_type<__half>(g, s);
    return rotary_type<float>(g, s);
}

}  // namespace ssd
