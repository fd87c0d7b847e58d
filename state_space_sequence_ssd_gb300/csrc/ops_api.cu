// ops_api.cu -- the C entries of the layer operators around the scan (short convolution, selective scan with one
// decay per channel and state entry, layer norm): argument validation, workspace and launch order.  Every exported
// function is declared and documented in include/ssd.h.
#include <cmath>

#include "ops.cuh"

using namespace ssd;

namespace {

uintptr_t size_of(int dtype) { return dtype == SSD_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == SSD_BF16 || dtype == SSD_F16 || dtype == SSD_F32; }

// Limits of the grids (one row of blocks in z per row; blocks of at least 32 tokens in y, or of 16 on rows that a rule holds
// short: kMaxGrid in ops.cuh, asserted beside the rules) and of 32-bit channel counts.
constexpr int kMaxBatch = kMaxGrid, kMaxTokens = kMaxGrid * 32, kMaxChannels = 1 << 20;

// Whether `batch` rows of `tokens` tokens of `channels` elements at these strides do not overlap.
bool apart(int64_t batch_stride, int64_t token_stride, int64_t batch, int64_t tokens, int64_t channels) {
    if (batch_stride < 0 || token_stride < 0) return false;
    const bool rows = tokens == 1 || token_stride >= channels, all = batch == 1 || batch_stride >= channels;
    return rows && all && (batch == 1 || tokens == 1 || batch_stride >= (tokens - 1) * token_stride + channels ||
                           token_stride >= (batch - 1) * batch_stride + channels);
}

int read_pieces(void* const (&p)[3], const int (&n)[3], const int (&f32)[3], int channels, uintptr_t size, Pieces* out) {
    int64_t sum = 0;
    for (int i = 0; i < 3; ++i) {
        if (n[i] < 0 || (n[i] > 0 && p[i] == nullptr)) return SSD_ERR_INVALID_ARG;
        if (n[i] > 0 && !aligned_to(p[i], f32[i] ? 4 : size)) return SSD_ERR_INVALID_ARG;
        if (i > 0 && n[i] > 0 && n[i - 1] == 0) return SSD_ERR_INVALID_ARG;
        sum += n[i];
        out->p[i] = n[i] > 0 ? p[i] : nullptr;
        out->n[i] = n[i];
        out->f32[i] = f32[i] != 0;
    }
    return sum == channels ? SSD_OK : SSD_ERR_INVALID_ARG;
}

int read_conv(int dtype, const void* x, int64_t x_batch, int64_t x_token, const float* weight, const float* bias,
              const void* init, const int* lengths, int batch, int seqlen, int channels, int width, int silu, ConvArgs* a) {
    if (!x || !weight || !known(dtype) || batch <= 0 || seqlen <= 0 || channels <= 0 || width <= 0 || x_batch < 0 ||
        x_token < 0)
        return SSD_ERR_INVALID_ARG;
    if (width < 2 || width > 4 || batch > kMaxBatch || seqlen > kMaxTokens || channels > kMaxChannels)
        return SSD_ERR_UNSUPPORTED;
    const uintptr_t size = size_of(dtype);
    if (!aligned_to(x, size) || !aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(init, size) ||
        !aligned_to(lengths, 4)) return SSD_ERR_INVALID_ARG;
    *a = ConvArgs{dtype, batch, seqlen, channels, width, silu != 0, x, x_batch, x_token, weight, bias, init, lengths};
    return SSD_OK;
}

int read_selective(int dtype, const void* x, const void* dt, const float* A, const void* B, const void* C, const float* D,
                   const float* init, const int* lengths, const ssd_selective_strides* given, int batch, int seqlen,
                   int channels, int ngroups, int dstate, const ssd_input_options* o, bool step, SelectiveArgs* a) {
    if (!x || !dt || !A || !B || !C || !known(dtype) || batch <= 0 || seqlen <= 0 || channels <= 0 || ngroups <= 0 ||
        dstate <= 0 || channels % ngroups != 0)
        return SSD_ERR_INVALID_ARG;
    if (dstate > 128 || batch > kMaxBatch || seqlen > kMaxTokens || channels > kMaxChannels) return SSD_ERR_UNSUPPORTED;
    const uintptr_t size = size_of(dtype);
    const void* z = o != nullptr ? o->z : nullptr;
    if (!aligned_to(x, size) || !aligned_to(dt, size) || !aligned_to(B, size) || !aligned_to(C, size) ||
        !aligned_to(z, size) || !aligned_to(A, 4) || !aligned_to(D, 4) ||
        !aligned_to(init, 4) || !aligned_to(lengths, 4))
        return SSD_ERR_INVALID_ARG;
    DtOpts dto;
    dto.lo = -INFINITY;  // no limits
    dto.hi = INFINITY;
    if (o != nullptr) {
        if (!aligned_to(o->dt_bias, 4)) return SSD_ERR_INVALID_ARG;
        if (o->dt_limit && !(o->dt_min <= o->dt_max)) return SSD_ERR_INVALID_ARG;  // also rejects a NaN bound
        dto.bias = o->dt_bias;
        dto.softplus = o->dt_softplus != 0;
        dto.limit = o->dt_limit != 0;
        if (dto.limit) {
            dto.lo = o->dt_min;
            dto.hi = o->dt_max;
        }
    }
    const int64_t row = channels, bc = (int64_t)ngroups * dstate;
    ssd_selective_strides s = {seqlen * row, row, seqlen * row, row, seqlen * row, row, seqlen * bc, bc, seqlen * bc, bc};
    if (given != nullptr) s = *given;
    if (step) s.x_token = s.dt_token = s.z_token = s.B_token = s.C_token = 0;  // not read
    if (z == nullptr) s.z_batch = s.z_token = 0;
    const long long all[] = {s.x_batch, s.x_token, s.dt_batch, s.dt_token, s.z_batch,
                             s.z_token, s.B_batch, s.B_token, s.C_batch, s.C_token};
    for (long long v : all)
        if (v < 0) return SSD_ERR_INVALID_ARG;
    *a = SelectiveArgs{dtype, batch, seqlen, channels, ngroups, dstate, x, dt, B, C, z,
                       s.x_batch, s.x_token, s.dt_batch, s.dt_token, s.B_batch, s.B_token,
                       s.C_batch, s.C_token, s.z_batch, s.z_token, A, D, init, lengths, dto};
    return SSD_OK;
}

// Gives `ws` back to the pool in stream order; an error of the launches comes first.
int give_back(void* ws, cudaStream_t s, int r) {
    if (ws != nullptr && cudaFreeAsync(ws, s) != cudaSuccess && r == SSD_OK) r = SSD_ERR_CUDA;
    return r;
}

}  // namespace

extern "C" {

int ssd_conv_forward(int dtype, const void* x, long long x_batch_stride, long long x_token_stride, const float* weight,
                     const float* bias, const void* init_state, const int* lengths, int batch, int seqlen, int channels,
                     int width, int silu, void* y0, int n0, void* y1, int n1, void* y2, int n2, void* final_state,
                     cudaStream_t stream) {
    ConvArgs a;
    int r = read_conv(dtype, x, x_batch_stride, x_token_stride, weight, bias, init_state, lengths, batch, seqlen, channels,
                      width, silu, &a);
    if (r != SSD_OK) return r;
    Pieces y;
    r = read_pieces({y0, y1, y2}, {n0, n1, n2}, {0, 0, 0}, channels, size_of(dtype), &y);
    if (r != SSD_OK) return r;
    if (!aligned_to(final_state, size_of(dtype))) return SSD_ERR_INVALID_ARG;
    return launch_conv_forward(a, y, final_state, stream);
}

int ssd_conv_backward(int dtype, const void* x, long long x_batch_stride, long long x_token_stride, const float* weight,
                      const float* bias, const void* init_state, const int* lengths, int batch, int seqlen, int channels,
                      int width, int silu, const void* dy0, int n0, int f32_0, const void* dy1, int n1, int f32_1,
                      const void* dy2, int n2, int f32_2, const void* dfinal, void* dx, long long dx_batch_stride,
                      long long dx_token_stride, float* dweight, float* dbias, void* dinit, cudaStream_t stream) {
    ConvArgs a;
    int r = read_conv(dtype, x, x_batch_stride, x_token_stride, weight, bias, init_state, lengths, batch, seqlen, channels,
                      width, silu, &a);
    if (r != SSD_OK) return r;
    Pieces dy;
    r = read_pieces({const_cast<void*>(dy0), const_cast<void*>(dy1), const_cast<void*>(dy2)}, {n0, n1, n2},
                    {f32_0, f32_1, f32_2}, channels, size_of(dtype), &dy);
    if (r != SSD_OK) return r;
    const uintptr_t size = size_of(dtype);
    if (!dx || !aligned_to(dx, size) || !aligned_to(dfinal, size) || !aligned_to(dinit, size) ||
        !aligned_to(dweight, 4) || !aligned_to(dbias, 4) ||
        !apart(dx_batch_stride, dx_token_stride, batch, seqlen, channels))
        return SSD_ERR_INVALID_ARG;
    void* ws = nullptr;
    const size_t bytes = (size_t)conv_backward_rows(a) * channels * (width + 1) * sizeof(float);
    if (take_workspace(&ws, bytes, stream) != SSD_OK) return SSD_ERR_NO_MEMORY;
    r = launch_conv_backward(a, dy, dfinal, dx, dx_batch_stride, dx_token_stride, dweight, dbias, dinit,
                             static_cast<float*>(ws), stream);
    return give_back(ws, stream, r);
}

int ssd_conv_step(int dtype, const void* x, long long x_row_stride, const float* weight, const float* bias, void* state,
                  const int* slots, int nslots, int batch, int channels, int width, int silu, void* y0, int n0, void* y1,
                  int n1, void* y2, int n2, cudaStream_t stream) {
    ConvArgs a;
    int r = read_conv(dtype, x, x_row_stride, 0, weight, bias, nullptr, nullptr, batch, 1, channels, width, silu, &a);
    if (r != SSD_OK) return r;
    Pieces y;
    r = read_pieces({y0, y1, y2}, {n0, n1, n2}, {0, 0, 0}, channels, size_of(dtype), &y);
    if (r != SSD_OK) return r;
    if (!state || !aligned_to(state, size_of(dtype)) || !aligned_to(slots, 4) || nslots <= 0 ||
        (slots == nullptr && nslots < batch))
        return SSD_ERR_INVALID_ARG;
    int* err = error_words();
    if (err == nullptr) return SSD_ERR_CUDA;
    return launch_conv_step(a, state, slots, nslots, y, err, stream);
}

int ssd_selective_forward(int dtype, const void* x, const void* dt, const float* A, const void* B, const void* C,
                          const float* D, const float* init_state, const int* lengths,
                          const ssd_selective_strides* strides, int batch, int seqlen, int channels, int ngroups,
                          int dstate, const ssd_input_options* options, void* y, float* final_state,
                          cudaStream_t stream) {
    SelectiveArgs a;
    int r = read_selective(dtype, x, dt, A, B, C, D, init_state, lengths, strides, batch, seqlen, channels, ngroups, dstate,
                           options, false, &a);
    if (r != SSD_OK) return r;
    if (!y || !aligned_to(y, size_of(dtype)) || !aligned_to(final_state, 4)) return SSD_ERR_INVALID_ARG;
    const SelectivePlan plan = selective_plan(a, multiprocessors());
    const size_t bytes = selective_workspace(a, plan);
    void* ws = nullptr;
    if (bytes > 0 && take_workspace(&ws, bytes, stream) != SSD_OK) return SSD_ERR_NO_MEMORY;
    r = launch_selective_forward(a, plan, y, final_state, static_cast<float*>(ws), stream);
    return give_back(ws, stream, r);
}

int ssd_selective_backward(int dtype, const void* x, const void* dt, const float* A, const void* B, const void* C,
                           const float* D, const float* init_state, const int* lengths,
                           const ssd_selective_strides* strides, int batch, int seqlen, int channels, int ngroups,
                           int dstate, const ssd_input_options* options, const void* dy, const float* dfinal, void* dx,
                           void* ddt, float* dA, float* dB, float* dC, float* dD, void* dz, float* ddt_bias,
                           float* dinit, cudaStream_t stream) {
    SelectiveArgs a;
    int r = read_selective(dtype, x, dt, A, B, C, D, init_state, lengths, strides, batch, seqlen, channels, ngroups, dstate,
                           options, false, &a);
    if (r != SSD_OK) return r;
    const uintptr_t size = size_of(dtype);
    if (!dy || !dx || !ddt || !dA || !dB || !dC || (a.z != nullptr) != (dz != nullptr)) return SSD_ERR_INVALID_ARG;
    if (!aligned_to(dy, size) || !aligned_to(dx, size) || !aligned_to(ddt, size) || !aligned_to(dz, size) ||
        !aligned_to(dA, 4) || !aligned_to(dB, 4) || !aligned_to(dC, 4) ||
        !aligned_to(dD, 4) || !aligned_to(ddt_bias, 4) || !aligned_to(dinit, 4) || !aligned_to(dfinal, 4))
        return SSD_ERR_INVALID_ARG;
    const SelectiveGrads g = {dy, dfinal, dx, ddt, dz, dA, dB, dC, dD, ddt_bias, dinit};
    void* ws = nullptr;
    if (take_workspace(&ws, selective_backward_workspace(a), stream) != SSD_OK) return SSD_ERR_NO_MEMORY;
    r = launch_selective_backward(a, g, static_cast<float*>(ws), stream);
    return give_back(ws, stream, r);
}

int ssd_selective_step(int dtype, const void* x, const void* dt, const float* A, const void* B, const void* C,
                       const float* D, float* state, const int* slots, int nslots, const ssd_selective_strides* strides,
                       int batch, int channels, int ngroups, int dstate, const ssd_input_options* options, void* y,
                       cudaStream_t stream) {
    SelectiveArgs a;
    const int r = read_selective(dtype, x, dt, A, B, C, D, nullptr, nullptr, strides, batch, 1, channels, ngroups, dstate,
                                 options, true, &a);
    if (r != SSD_OK) return r;
    if (!y || !aligned_to(y, size_of(dtype)) || !state || !aligned_to(state, 4) || !aligned_to(slots, 4) ||
        nslots <= 0 ||
        (slots == nullptr && nslots < batch))
        return SSD_ERR_INVALID_ARG;
    int* err = error_words();
    if (err == nullptr) return SSD_ERR_CUDA;
    return launch_selective_step(a, state, slots, nslots, y, err, stream);
}

int ssd_layer_norm_forward(int dtype, const void* x, long long x_row_stride, const float* weight, const float* bias,
                           float eps, long long rows, int width, void* y, float* mean, float* rstd,
                           cudaStream_t stream) {
    if (!x || !y || !known(dtype) || rows <= 0 || width <= 0 || x_row_stride < 0 || !(eps >= 0.f) || std::isinf(eps))
        return SSD_ERR_INVALID_ARG;
    if (width > kMaxChannels) return SSD_ERR_UNSUPPORTED;
    const uintptr_t size = size_of(dtype);
    if (!aligned_to(x, size) || !aligned_to(y, size) || !aligned_to(weight, 4) || !aligned_to(bias, 4) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return SSD_ERR_INVALID_ARG;
    return launch_layer_norm_forward(dtype, x, x_row_stride, weight, bias, eps, rows, width, y, mean, rstd, stream);
}

int ssd_layer_norm_backward(int dtype, const void* x, long long x_row_stride, const float* weight, const float* mean,
                            const float* rstd, const void* dy, long long dy_row_stride, long long rows, int width,
                            void* dx, float* dweight, float* dbias, cudaStream_t stream) {
    if (!x || !mean || !rstd || !dy || !dx || !known(dtype) || rows <= 0 || width <= 0 || x_row_stride < 0 ||
        dy_row_stride < 0)
        return SSD_ERR_INVALID_ARG;
    if (width > kMaxChannels) return SSD_ERR_UNSUPPORTED;
    const uintptr_t size = size_of(dtype);
    if (!aligned_to(x, size) || !aligned_to(dy, size) || !aligned_to(dx, size) || !aligned_to(weight, 4) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
        !aligned_to(dweight, 4) || !aligned_to(dbias, 4))
        return SSD_ERR_INVALID_ARG;
    const int parts = layer_norm_parts(rows, multiprocessors());
    void* ws = nullptr;
    if ((dweight != nullptr || dbias != nullptr) &&
        take_workspace(&ws, (size_t)parts * 2 * width * sizeof(float), stream) != SSD_OK)
        return SSD_ERR_NO_MEMORY;
    const int r = launch_layer_norm_backward(dtype, x, x_row_stride, weight, mean, rstd, dy, dy_row_stride, rows, width, dx,
                                             dweight, dbias, static_cast<float*>(ws), parts, stream);
    return give_back(ws, stream, r);
}

}  // extern "C"
