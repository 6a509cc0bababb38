// kda_api_mixer.cu -- C-ABI front end of the operators around the recurrence: convolution, q/k norm and
// rotation, selective scan. Argument validation and kernel dispatch.
#include <cuda_runtime.h>

#include <math.h>

#include "../../include/kda.h"
#include "kda_conv.h"
#include "kda_qk.h"
#include "kda_scan.h"

static_assert(KDA_NORM_NONE == kda::kNormNone && KDA_NORM_L2 == kda::kNormL2 && KDA_NORM_RMS == kda::kNormRms,
              "norm kinds");

namespace {

constexpr int64_t kMaxElements = int64_t(1) << 40;   // element offsets stay well inside 64 bits

bool aligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned16(const void *p) { return aligned(p, 16); }
bool float_or_bf16(kda_dtype d) { return d == KDA_DTYPE_BF16 || d == KDA_DTYPE_FP32; }
int64_t size_of(kda_dtype d) { return d == KDA_DTYPE_FP32 ? 4 : 2; }

// rows of `width` bytes, `stride` bytes apart
struct Span {
    const void *p;
    int64_t rows, width, stride;
};
Span whole(const void *p, int64_t bytes) { return {p, 1, bytes, bytes}; }
Span offsets(const kda::Seqs &s) { return whole(s.cu, (static_cast<int64_t>(s.n) + 1) * 4); }

// Whether two buffers share a byte. Rows with the same stride may be interleaved (slices of one
// tensor's columns): those share none where their columns do not meet.
bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t ea = pa + static_cast<uintptr_t>((a.rows - 1) * a.stride + a.width);
    const uintptr_t eb = pb + static_cast<uintptr_t>((b.rows - 1) * b.stride + b.width);
    if (pa >= eb || pb >= ea) return false;
    if (a.stride == b.stride && a.rows > 1 && b.rows > 1) {
        const int64_t s = a.stride;
        const int64_t off = pb >= pa ? static_cast<int64_t>((pb - pa) % static_cast<uintptr_t>(s))
                                     : (s - static_cast<int64_t>((pa - pb) % static_cast<uintptr_t>(s))) % s;
        // b's columns start `off` bytes into a's rows
        if (off >= a.width && off + b.width <= s) return false;
    }
    return true;
}
bool same(const Span &a, const Span &b) {
    return a.p == b.p && a.width == b.width && (a.stride == b.stride || (a.rows <= 1 && b.rows <= 1));
}
template <int NO, int NI>
bool any_overlap(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return true;
        for (int j = 0; j < NI; ++j)
            if (overlap(outs[i], ins[j])) return true;
    }
    return false;
}

kda_status check_device() {
    int dev = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return KDA_ERR_CUDA;
    return major == 10 ? KDA_OK : KDA_ERR_UNSUPPORTED_DEVICE;
}

kda_status done(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

kda_status check_sequences(const int32_t *cu, int32_t num_seqs, int32_t batch, int64_t seq_len, kda::Seqs *s, int64_t *rows) {
    if (batch < 0 || seq_len < 0 || num_seqs < 0) return KDA_ERR_BAD_SHAPE;
    if (cu && batch != 1) return KDA_ERR_VARLEN_BATCH;
    if (!aligned(cu, 4)) return KDA_ERR_BAD_ALIGNMENT;
    if (seq_len > kMaxElements / (batch > 1 ? batch : 1)) return KDA_ERR_TOO_LARGE;   // before their product is formed
    s->cu = cu;
    s->n = cu ? num_seqs : batch;
    s->len = seq_len;
    // without sequences there are no tokens either: the kernels look every token's sequence up
    *rows = s->n == 0 ? 0 : cu ? seq_len : static_cast<int64_t>(batch) * seq_len;
    return KDA_OK;
}

// a row stride in elements of `size` bytes: rows do not overlap, and each starts on 16 bytes
kda_status check_stride(int64_t rows, int64_t stride, int64_t width, int64_t size) {
    if (rows <= 1) return KDA_OK;
    if (stride < width) return KDA_ERR_BAD_SHAPE;
    if ((stride * size) & 15) return KDA_ERR_BAD_ALIGNMENT;
    return rows > kMaxElements / stride ? KDA_ERR_TOO_LARGE : KDA_OK;
}

#define KDA_TRY(call)                          \
    do {                                       \
        const kda_status st_ = (call);         \
        if (st_ != KDA_OK) return st_;         \
    } while (0)

// ---------------------------------------------------------------- convolution

kda_status conv_args(const void *x, kda_dtype dtype, int64_t x_stride, const float *weight, const float *bias,
                     uint32_t flags, int64_t rows, int32_t channels, int32_t taps) {
    if (flags & ~static_cast<uint32_t>(KDA_FLAG_CONV_SILU)) return KDA_ERR_BAD_OPTION;
    if (channels < 8 || channels % 8 || taps < kda::kConvMinTaps || taps > kda::kConvMaxTaps) return KDA_ERR_BAD_SHAPE;
    if (!float_or_bf16(dtype)) return KDA_ERR_DTYPE;
    if (rows > 0 && (!x || !weight)) return KDA_ERR_NULL_PTR;
    if (!aligned16(x) || !aligned16(weight) || !aligned(bias, 4)) return KDA_ERR_BAD_ALIGNMENT;
    if (rows > kMaxElements / channels) return KDA_ERR_TOO_LARGE;
    return check_stride(rows, x_stride, channels, size_of(dtype));
}

// ---------------------------------------------------------------- q/k

kda_status qk_args(const void *q, int64_t q_stride, const void *k, int64_t k_stride, int64_t rows, int32_t q_heads,
                   int32_t k_heads, int32_t head_dim, int32_t norm, float eps, const float *q_weight,
                   const float *k_weight, const int32_t *positions, const float *inv_freq, int32_t rot_dim,
                   float factor, kda::QkParams *p) {
    if (norm != KDA_NORM_NONE && norm != KDA_NORM_L2 && norm != KDA_NORM_RMS) return KDA_ERR_BAD_OPTION;
    if (!(eps >= 0.f) || !isfinite(eps) || !isfinite(factor)) return KDA_ERR_BAD_OPTION;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KDA_ERR_BAD_SHAPE;
    if (rows < 0 || q_heads < 1 || k_heads < 0) return KDA_ERR_BAD_SHAPE;
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16) return KDA_ERR_BAD_SHAPE;
    if (q_heads > (1 << 20) || k_heads > (1 << 20)) return KDA_ERR_TOO_LARGE;
    if (rows > 0 && (!q || (k_heads && !k) || (rot_dim && (!positions || !inv_freq)))) return KDA_ERR_NULL_PTR;
    if (!aligned16(q) || !aligned16(k) || !aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(positions, 4) ||
        !aligned(inv_freq, 4))
        return KDA_ERR_BAD_ALIGNMENT;
    if (rows > kMaxElements / (static_cast<int64_t>(q_heads + k_heads) * head_dim)) return KDA_ERR_TOO_LARGE;
    KDA_TRY(check_stride(rows, q_stride, static_cast<int64_t>(q_heads) * head_dim, 2));
    if (k_heads) KDA_TRY(check_stride(rows, k_stride, static_cast<int64_t>(k_heads) * head_dim, 2));
    p->rows = rows;
    p->Hq = q_heads;
    p->Hk = k_heads;
    p->D = head_dim;
    p->norm = norm;
    p->eps = eps;
    p->q_weight = q_weight;
    p->k_weight = k_weight;
    p->positions = positions;
    p->inv_freq = inv_freq;
    p->rot = rot_dim;
    p->factor = factor;
    p->q = static_cast<const uint16_t *>(q);
    p->k = static_cast<const uint16_t *>(k);
    p->q_stride = q_stride;
    p->k_stride = k_stride;
    return KDA_OK;
}

// ---------------------------------------------------------------- scan

struct ScanArgs {
    const void *x;
    int64_t x_stride;
    const float *dt, *A;
    const void *B;
    int64_t b_stride;
    const void *C;
    int64_t c_stride;
    const float *D, *dt_bias;
    uint32_t flags;
    int32_t H, G, P, N;
};

kda_status scan_args(const ScanArgs &a, int64_t rows) {
    if (a.flags & ~static_cast<uint32_t>(KDA_FLAG_SCAN_SOFTPLUS)) return KDA_ERR_BAD_OPTION;
    if ((a.P != 64 && a.P != 128) || (a.N != 64 && a.N != 128)) return KDA_ERR_BAD_SHAPE;
    if (a.H < 1 || a.G < 1 || a.H % a.G) return KDA_ERR_BAD_SHAPE;
    if (rows > 0 && (!a.x || !a.dt || !a.A || !a.B || !a.C)) return KDA_ERR_NULL_PTR;
    if (!aligned16(a.x) || !aligned16(a.B) || !aligned16(a.C) || !aligned(a.dt, 4) || !aligned(a.A, 4) ||
        !aligned(a.D, 4) || !aligned(a.dt_bias, 4))
        return KDA_ERR_BAD_ALIGNMENT;
    if (a.H > (1 << 20) || rows > kMaxElements / (static_cast<int64_t>(a.H) * a.P) ||
        rows > kMaxElements / (static_cast<int64_t>(a.G) * a.N))
        return KDA_ERR_TOO_LARGE;
    KDA_TRY(check_stride(rows, a.x_stride, static_cast<int64_t>(a.H) * a.P, 2));
    KDA_TRY(check_stride(rows, a.b_stride, static_cast<int64_t>(a.G) * a.N, 2));
    return check_stride(rows, a.c_stride, static_cast<int64_t>(a.G) * a.N, 2);
}

void scan_params(const ScanArgs &a, const kda::Seqs &s, int64_t rows, kda::ScanParams *p) {
    *p = kda::ScanParams();
    p->seqs = s;
    p->rows = rows;
    p->H = a.H;
    p->G = a.G;
    p->P = a.P;
    p->N = a.N;
    p->x = static_cast<const uint16_t *>(a.x);
    p->x_stride = a.x_stride;
    p->dt = a.dt;
    p->A = a.A;
    p->B = static_cast<const uint16_t *>(a.B);
    p->C = static_cast<const uint16_t *>(a.C);
    p->b_stride = a.b_stride;
    p->c_stride = a.c_stride;
    p->D = a.D;
    p->dt_bias = a.dt_bias;
    p->softplus = (a.flags & KDA_FLAG_SCAN_SOFTPLUS) != 0;
}

bool scan_too_large(int64_t rows, int64_t n, int32_t H, int32_t P) {
    // rows are 32-bit coordinates of tensor maps; the largest grid is one CTA per (64-token cell, head, 64 columns)
    if (rows > 0x7fffffffLL) return true;
    return 2 * kda::scan_cells(rows, n) > 0x7fffffffLL / (static_cast<int64_t>(H) * (P / 64));
}

// the gradients': the kept states' rows, too, are 32-bit coordinates
bool scan_bwd_too_large(int64_t rows, int64_t n, int32_t H, int32_t P, int32_t N) {
    return scan_too_large(rows, n, H, P) || kda::scan_cells(rows, n) > 0x7fffffffLL / (static_cast<int64_t>(H) * N);
}

kda_status check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return KDA_OK;
    if (!ws) return KDA_ERR_NULL_PTR;
    if (!aligned(ws, 256)) return KDA_ERR_BAD_ALIGNMENT;
    return have < need ? KDA_ERR_WORKSPACE : KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_conv_fwd(const void *x, kda_dtype dtype, int64_t x_stride, const float *weight, const float *bias,
                        uint32_t flags, const int32_t *cu_seqlens, int32_t num_seqs, int32_t batch, int64_t seq_len,
                        int32_t channels, int32_t taps, const void *initial_state, void *final_state, void *out,
                        int64_t out_stride, kda_stream_t stream) {
    kda::ConvParams p = {};
    KDA_TRY(check_sequences(cu_seqlens, num_seqs, batch, seq_len, &p.seqs, &p.rows));
    KDA_TRY(conv_args(x, dtype, x_stride, weight, bias, flags, p.rows, channels, taps));
    if (p.rows > 0 && !out) return KDA_ERR_NULL_PTR;
    if (!aligned16(out) || !aligned16(initial_state) || !aligned16(final_state)) return KDA_ERR_BAD_ALIGNMENT;
    const int64_t e = size_of(dtype), row = channels * e, st = static_cast<int64_t>(p.seqs.n) * (taps - 1) * row;
    KDA_TRY(check_stride(p.rows, out_stride, channels, e));
    const Span outs[] = {{out, p.rows, row, out_stride * e}, whole(final_state, st)};
    const Span ins[] = {{x, p.rows, row, x_stride * e}, whole(initial_state, st), whole(weight, 4LL * channels * taps),
                        whole(bias, channels * 4LL), offsets(p.seqs)};
    if (any_overlap(outs, ins)) return KDA_ERR_OVERLAP;
    if (p.seqs.n == 0) return KDA_OK;
    KDA_TRY(check_device());
    p.C = channels;
    p.W = taps;
    p.fp32 = dtype == KDA_DTYPE_FP32;
    p.silu = (flags & KDA_FLAG_CONV_SILU) != 0;
    p.weight = weight;
    p.bias = bias;
    p.x = x;
    p.x_stride = x_stride;
    p.init = initial_state;
    p.out = out;
    p.out_stride = out_stride;
    p.final_state = final_state;
    return done(kda::launch_conv_fwd(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_conv_bwd_workspace(int64_t total_tokens, int32_t channels, int32_t taps) {
    if (total_tokens < 0 || channels < 8 || channels % 8 || taps < kda::kConvMinTaps || taps > kda::kConvMaxTaps ||
        total_tokens > kMaxElements / channels)
        return 0;
    return static_cast<size_t>(kda::conv_bwd_blocks(total_tokens, channels)) * (taps + 1) * channels * sizeof(float);
}

kda_status kda_conv_bwd(const void *x, kda_dtype dtype, int64_t x_stride, const float *weight, const float *bias,
                        uint32_t flags, const int32_t *cu_seqlens, int32_t num_seqs, int32_t batch, int64_t seq_len,
                        int32_t channels, int32_t taps, const void *initial_state, const void *dout,
                        kda_dtype dout_dtype, int64_t dout_stride, const void *dfinal_state, void *dx,
                        int64_t dx_stride, float *dweight, float *dbias, void *dinitial_state, void *workspace,
                        size_t workspace_bytes, kda_stream_t stream) {
    kda::ConvParams p = {};
    KDA_TRY(check_sequences(cu_seqlens, num_seqs, batch, seq_len, &p.seqs, &p.rows));
    KDA_TRY(conv_args(x, dtype, x_stride, weight, bias, flags, p.rows, channels, taps));
    // a bf16 x takes a gradient of either type, an fp32 x an fp32 one
    if (!float_or_bf16(dout_dtype) || (dtype == KDA_DTYPE_FP32 && dout_dtype != KDA_DTYPE_FP32)) return KDA_ERR_DTYPE;
    if (p.rows > 0 && (!dout || !dx)) return KDA_ERR_NULL_PTR;
    if (!weight) return KDA_ERR_NULL_PTR;
    if (!aligned16(dout) || !aligned16(dx) || !aligned16(initial_state) || !aligned16(dfinal_state) ||
        !aligned16(dinitial_state) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return KDA_ERR_BAD_ALIGNMENT;
    const int64_t e = size_of(dtype), ed = size_of(dout_dtype), row = channels * e;
    const int64_t st = static_cast<int64_t>(p.seqs.n) * (taps - 1) * row;
    KDA_TRY(check_stride(p.rows, dout_stride, channels, ed));
    KDA_TRY(check_stride(p.rows, dx_stride, channels, e));
    const size_t need = kda_conv_bwd_workspace(p.rows, channels, taps);
    KDA_TRY(check_workspace(workspace, workspace_bytes, need));
    const Span outs[] = {{dx, p.rows, row, dx_stride * e}, whole(dweight, 4LL * channels * taps),
                         whole(dbias, channels * 4LL), whole(dinitial_state, st),
                         whole(workspace, static_cast<int64_t>(need))};
    const Span ins[] = {{x, p.rows, row, x_stride * e}, {dout, p.rows, channels * ed, dout_stride * ed},
                        whole(weight, 4LL * channels * taps), whole(bias, channels * 4LL), whole(initial_state, st),
                        whole(dfinal_state, st), offsets(p.seqs)};
    if (any_overlap(outs, ins)) return KDA_ERR_OVERLAP;
    KDA_TRY(check_device());
    p.C = channels;
    p.W = taps;
    p.fp32 = dtype == KDA_DTYPE_FP32;
    p.silu = (flags & KDA_FLAG_CONV_SILU) != 0;
    p.weight = weight;
    p.bias = bias;
    p.x = x;
    p.x_stride = x_stride;
    p.init = initial_state;
    p.dout = dout;
    p.dout_stride = dout_stride;
    p.dout_fp32 = dout_dtype == KDA_DTYPE_FP32;
    p.dfinal = dfinal_state;
    p.dx = dx;
    p.dx_stride = dx_stride;
    p.dinit = dinitial_state;
    p.dweight = dweight;
    p.dbias = dbias;
    p.partial = static_cast<float *>(workspace);
    return done(kda::launch_conv_bwd(p, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_conv_decode(const void *x, kda_dtype dtype, int64_t x_stride, const float *weight, const float *bias,
                           uint32_t flags, int32_t batch, int32_t channels, int32_t taps, const void *state_in,
                           void *state_out, void *out, int64_t out_stride, kda_stream_t stream) {
    if (batch < 0) return KDA_ERR_BAD_SHAPE;
    KDA_TRY(conv_args(x, dtype, x_stride, weight, bias, flags, batch, channels, taps));
    if (batch > 0 && !out) return KDA_ERR_NULL_PTR;
    if (!aligned16(out) || !aligned16(state_in) || !aligned16(state_out)) return KDA_ERR_BAD_ALIGNMENT;
    const int64_t e = size_of(dtype), row = channels * e, st = static_cast<int64_t>(batch) * (taps - 1) * row;
    KDA_TRY(check_stride(batch, out_stride, channels, e));
    if (state_in != state_out && overlap(whole(state_in, st), whole(state_out, st))) return KDA_ERR_STATE_OVERLAP;
    const Span outs[] = {{out, batch, row, out_stride * e}, whole(state_out, st)};
    const Span ins[] = {{x, batch, row, x_stride * e}, whole(weight, 4LL * channels * taps), whole(bias, channels * 4LL)};
    if (any_overlap(outs, ins) || overlap(outs[0], whole(state_in, st))) return KDA_ERR_OVERLAP;
    if (batch == 0) return KDA_OK;
    KDA_TRY(check_device());
    kda::ConvDecodeParams p = {};
    p.batch = batch;
    p.C = channels;
    p.W = taps;
    p.fp32 = dtype == KDA_DTYPE_FP32;
    p.silu = (flags & KDA_FLAG_CONV_SILU) != 0;
    p.weight = weight;
    p.bias = bias;
    p.x = x;
    p.x_stride = x_stride;
    p.state_in = state_in;
    p.state_out = state_out;
    p.out = out;
    p.out_stride = out_stride;
    return done(kda::launch_conv_decode(p, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_qk_fwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride, int64_t rows, int32_t q_heads,
                      int32_t k_heads, int32_t head_dim, int32_t norm, float eps, const float *q_weight,
                      const float *k_weight, const int32_t *positions, const float *inv_freq, int32_t rot_dim,
                      int32_t interleaved, float factor, void *q_out, int64_t q_out_stride, void *k_out,
                      int64_t k_out_stride, kda_stream_t stream) {
    kda::QkParams p = {};
    KDA_TRY(qk_args(q, q_stride, k, k_stride, rows, q_heads, k_heads, head_dim, norm, eps, q_weight, k_weight,
                    positions, inv_freq, rot_dim, factor, &p));
    if (rows > 0 && (!q_out || (k_heads && !k_out))) return KDA_ERR_NULL_PTR;
    if (!aligned16(q_out) || !aligned16(k_out)) return KDA_ERR_BAD_ALIGNMENT;
    const int64_t wq = static_cast<int64_t>(q_heads) * head_dim, wk = static_cast<int64_t>(k_heads) * head_dim;
    KDA_TRY(check_stride(rows, q_out_stride, wq, 2));
    if (k_heads) KDA_TRY(check_stride(rows, k_out_stride, wk, 2));
    // in place is fine: a head is read whole before it is written
    const Span qi = {q, rows, wq * 2, q_stride * 2}, ki = {k, rows, wk * 2, k_stride * 2};
    const Span qo = {q_out, rows, wq * 2, q_out_stride * 2}, ko = {k_out, rows, wk * 2, k_out_stride * 2};
    if ((overlap(qi, qo) && !same(qi, qo)) || (overlap(ki, ko) && !same(ki, ko)) || overlap(qi, ko) ||
        overlap(ki, qo) || overlap(qo, ko))
        return KDA_ERR_OVERLAP;
    const Span outs[] = {qo, ko};
    const Span ins[] = {whole(q_weight, head_dim * 4LL), whole(k_weight, head_dim * 4LL),
                        whole(positions, rot_dim ? rows * 4 : 0), whole(inv_freq, rot_dim * 2LL)};
    if (any_overlap(outs, ins)) return KDA_ERR_OVERLAP;
    if (rows == 0) return KDA_OK;
    KDA_TRY(check_device());
    p.interleaved = interleaved != 0;
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_out = static_cast<uint16_t *>(k_out);
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    return done(kda::launch_qk_fwd(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_qk_bwd_workspace(int64_t rows, int32_t q_heads, int32_t k_heads, int32_t head_dim) {
    if (rows < 0 || q_heads < 1 || k_heads < 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256)) return 0;
    if (q_heads > (1 << 20) || k_heads > (1 << 20) ||
        rows > kMaxElements / (static_cast<int64_t>(q_heads + k_heads) * head_dim))
        return 0;
    return static_cast<size_t>(kda::qk_bwd_blocks(rows, q_heads + k_heads, head_dim)) * 2 * head_dim * sizeof(float);
}

kda_status kda_qk_bwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride, int64_t rows, int32_t q_heads,
                      int32_t k_heads, int32_t head_dim, int32_t norm, float eps, const float *q_weight,
                      const float *k_weight, const int32_t *positions, const float *inv_freq, int32_t rot_dim,
                      int32_t interleaved, float factor, const void *dq_out, int64_t dq_out_stride,
                      const void *dk_out, int64_t dk_out_stride, kda_dtype dout_dtype, void *dq, int64_t dq_stride,
                      void *dk, int64_t dk_stride, float *dq_weight, float *dk_weight, void *workspace,
                      size_t workspace_bytes, kda_stream_t stream) {
    kda::QkParams p = {};
    KDA_TRY(qk_args(q, q_stride, k, k_stride, rows, q_heads, k_heads, head_dim, norm, eps, q_weight, k_weight,
                    positions, inv_freq, rot_dim, factor, &p));
    if (!float_or_bf16(dout_dtype)) return KDA_ERR_DTYPE;
    if (rows > 0 && (!dq_out || !dq || (k_heads && (!dk_out || !dk)))) return KDA_ERR_NULL_PTR;
    if (!aligned16(dq_out) || !aligned16(dk_out) || !aligned16(dq) || !aligned16(dk) || !aligned(dq_weight, 4) ||
        !aligned(dk_weight, 4))
        return KDA_ERR_BAD_ALIGNMENT;
    const int64_t wq = static_cast<int64_t>(q_heads) * head_dim, wk = static_cast<int64_t>(k_heads) * head_dim;
    const int64_t ed = size_of(dout_dtype);
    KDA_TRY(check_stride(rows, dq_out_stride, wq, ed));
    KDA_TRY(check_stride(rows, dq_stride, wq, 2));
    if (k_heads) {
        KDA_TRY(check_stride(rows, dk_out_stride, wk, ed));
        KDA_TRY(check_stride(rows, dk_stride, wk, 2));
    }
    const size_t need = dq_weight || dk_weight ? kda_qk_bwd_workspace(rows, q_heads, k_heads, head_dim) : 0;
    KDA_TRY(check_workspace(workspace, workspace_bytes, need));
    const Span outs[] = {{dq, rows, wq * 2, dq_stride * 2}, {dk, rows, wk * 2, dk_stride * 2},
                         whole(dq_weight, head_dim * 4LL), whole(dk_weight, head_dim * 4LL),
                         whole(need ? workspace : nullptr, static_cast<int64_t>(need))};
    const Span ins[] = {{q, rows, wq * 2, q_stride * 2}, {k, rows, wk * 2, k_stride * 2},
                        {dq_out, rows, wq * ed, dq_out_stride * ed}, {dk_out, rows, wk * ed, dk_out_stride * ed},
                        whole(q_weight, head_dim * 4LL), whole(k_weight, head_dim * 4LL),
                        whole(positions, rot_dim ? rows * 4 : 0), whole(inv_freq, rot_dim * 2LL)};
    if (any_overlap(outs, ins)) return KDA_ERR_OVERLAP;
    if (rows == 0 && !need) return KDA_OK;
    KDA_TRY(check_device());
    p.interleaved = interleaved != 0;
    p.q_out = static_cast<uint16_t *>(dq);
    p.k_out = static_cast<uint16_t *>(dk);
    p.q_out_stride = dq_stride;
    p.k_out_stride = dk_stride;
    p.dq_out = dq_out;
    p.dk_out = dk_out;
    p.dq_stride = dq_out_stride;
    p.dk_stride = dk_out_stride;
    p.dout_fp32 = dout_dtype == KDA_DTYPE_FP32;
    p.dq_weight = dq_weight;
    p.dk_weight = dk_weight;
    p.partial = need ? static_cast<float *>(workspace) : nullptr;
    return done(kda::launch_qk_bwd(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_scan_fwd_workspace(int64_t total_tokens, int32_t num_seqs, int32_t num_heads, int32_t head_dim,
                              int32_t state_dim) {
    if (total_tokens < 0 || num_seqs < 0 || num_heads < 1 || (head_dim != 64 && head_dim != 128) ||
        (state_dim != 64 && state_dim != 128) || num_heads > (1 << 20) ||
        total_tokens > kMaxElements / (static_cast<int64_t>(num_heads) * head_dim) ||
        scan_too_large(total_tokens, num_seqs, num_heads, head_dim))
        return 0;
    return kda::scan_fwd_workspace_bytes(total_tokens, num_seqs, num_heads, head_dim, state_dim);
}

kda_status kda_scan_fwd(const void *x, int64_t x_stride, const float *dt, const float *A, const void *B,
                        int64_t b_stride, const void *C, int64_t c_stride, const float *D, const float *dt_bias,
                        uint32_t flags, const int32_t *cu_seqlens, int32_t num_seqs, int32_t batch, int64_t seq_len,
                        int32_t num_heads, int32_t num_groups, int32_t head_dim, int32_t state_dim,
                        const void *initial_state, kda_dtype initial_dtype, void *final_state, kda_dtype final_dtype,
                        void *out, int64_t out_stride, void *workspace, size_t workspace_bytes, kda_stream_t stream) {
    kda::Seqs s = {};
    int64_t rows = 0;
    KDA_TRY(check_sequences(cu_seqlens, num_seqs, batch, seq_len, &s, &rows));
    const ScanArgs a = {x, x_stride, dt, A, B, b_stride, C, c_stride, D, dt_bias, flags,
                        num_heads, num_groups, head_dim, state_dim};
    KDA_TRY(scan_args(a, rows));
    if (initial_state && !float_or_bf16(initial_dtype)) return KDA_ERR_STATE_DTYPE;
    if (final_state && !float_or_bf16(final_dtype)) return KDA_ERR_STATE_DTYPE;
    if (initial_state && final_state && initial_dtype != final_dtype) return KDA_ERR_STATE_DTYPE;
    if (rows > 0 && !out) return KDA_ERR_NULL_PTR;
    if (s.n > 0 && !A) return KDA_ERR_NULL_PTR;
    if (!aligned16(out) || !aligned16(initial_state) || !aligned16(final_state)) return KDA_ERR_BAD_ALIGNMENT;
    KDA_TRY(check_stride(rows, out_stride, static_cast<int64_t>(num_heads) * head_dim, 2));
    if (scan_too_large(rows, s.n, num_heads, head_dim)) return KDA_ERR_TOO_LARGE;
    const size_t need = kda::scan_fwd_workspace_bytes(rows, s.n, num_heads, head_dim, state_dim);
    KDA_TRY(check_workspace(workspace, workspace_bytes, need));
    const int64_t wx = static_cast<int64_t>(num_heads) * head_dim * 2, wb = static_cast<int64_t>(num_groups) * state_dim * 2;
    const int64_t st = static_cast<int64_t>(s.n) * num_heads * state_dim * head_dim;
    const Span hi = whole(initial_state, st * size_of(initial_dtype)), ho = whole(final_state, st * size_of(final_dtype));
    if (overlap(hi, ho) && !same(hi, ho)) return KDA_ERR_STATE_OVERLAP;
    const Span outs[] = {{out, rows, wx, out_stride * 2}, ho, whole(need ? workspace : nullptr, static_cast<int64_t>(need))};
    const Span ins[] = {{x, rows, wx, x_stride * 2}, {B, rows, wb, b_stride * 2}, {C, rows, wb, c_stride * 2},
                        whole(dt, rows * num_heads * 4), whole(A, num_heads * 4LL), whole(D, num_heads * 4LL),
                        whole(dt_bias, num_heads * 4LL), offsets(s)};
    if (any_overlap(outs, ins) || overlap(outs[0], hi) || overlap(outs[2], hi)) return KDA_ERR_OVERLAP;
    if (s.n == 0) return KDA_OK;
    KDA_TRY(check_device());
    kda::ScanParams p;
    scan_params(a, s, rows, &p);
    p.h0 = initial_state;
    p.h0_fp32 = initial_dtype == KDA_DTYPE_FP32;
    p.hT = final_state;
    p.hT_fp32 = final_dtype == KDA_DTYPE_FP32;
    p.out = static_cast<uint16_t *>(out);
    p.out_stride = out_stride;
    p.ws = need ? static_cast<float *>(workspace) : nullptr;
    return done(kda::launch_scan_fwd(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_scan_bwd_workspace(int64_t total_tokens, int32_t num_seqs, int32_t num_heads, int32_t num_groups,
                              int32_t head_dim, int32_t state_dim) {
    if (total_tokens < 0 || num_seqs < 0 || num_heads < 1 || num_groups < 1 || num_heads % num_groups ||
        (head_dim != 64 && head_dim != 128) || (state_dim != 64 && state_dim != 128) || num_heads > (1 << 20) ||
        total_tokens > kMaxElements / (static_cast<int64_t>(num_heads) * head_dim) ||
        scan_bwd_too_large(total_tokens, num_seqs, num_heads, head_dim, state_dim))
        return 0;
    return kda::scan_bwd_workspace_bytes(total_tokens, num_seqs, num_heads, num_groups, head_dim, state_dim);
}

kda_status kda_scan_bwd(const void *x, int64_t x_stride, const float *dt, const float *A, const void *B,
                        int64_t b_stride, const void *C, int64_t c_stride, const float *D, const float *dt_bias,
                        uint32_t flags, const int32_t *cu_seqlens, int32_t num_seqs, int32_t batch, int64_t seq_len,
                        int32_t num_heads, int32_t num_groups, int32_t head_dim, int32_t state_dim,
                        const void *initial_state, kda_dtype initial_dtype, const void *dout, int64_t dout_stride,
                        const float *dfinal_state, void *dx, int64_t dx_stride, float *ddt, float *dA, void *dB,
                        int64_t db_stride, void *dC, int64_t dc_stride, float *dD, float *ddt_bias,
                        float *dinitial_state, void *workspace, size_t workspace_bytes, kda_stream_t stream) {
    kda::Seqs s = {};
    int64_t rows = 0;
    KDA_TRY(check_sequences(cu_seqlens, num_seqs, batch, seq_len, &s, &rows));
    const ScanArgs a = {x, x_stride, dt, A, B, b_stride, C, c_stride, D, dt_bias, flags,
                        num_heads, num_groups, head_dim, state_dim};
    KDA_TRY(scan_args(a, rows));
    if (initial_state && !float_or_bf16(initial_dtype)) return KDA_ERR_STATE_DTYPE;
    if (!A || !dA || (rows > 0 && (!dout || !dx || !ddt || !dB || !dC))) return KDA_ERR_NULL_PTR;
    if (!aligned16(dout) || !aligned16(dx) || !aligned16(dB) || !aligned16(dC) || !aligned16(initial_state) ||
        !aligned16(dfinal_state) || !aligned16(dinitial_state) || !aligned(ddt, 4) || !aligned(dA, 4) ||
        !aligned(dD, 4) || !aligned(ddt_bias, 4))
        return KDA_ERR_BAD_ALIGNMENT;
    const int64_t hp = static_cast<int64_t>(num_heads) * head_dim, gn = static_cast<int64_t>(num_groups) * state_dim;
    KDA_TRY(check_stride(rows, dout_stride, hp, 2));
    KDA_TRY(check_stride(rows, dx_stride, hp, 2));
    KDA_TRY(check_stride(rows, db_stride, gn, 2));
    KDA_TRY(check_stride(rows, dc_stride, gn, 2));
    if (scan_bwd_too_large(rows, s.n, num_heads, head_dim, state_dim)) return KDA_ERR_TOO_LARGE;
    const size_t need = kda::scan_bwd_workspace_bytes(rows, s.n, num_heads, num_groups, head_dim, state_dim);
    KDA_TRY(check_workspace(workspace, workspace_bytes, need));
    const int64_t st = static_cast<int64_t>(s.n) * num_heads * state_dim * head_dim;
    const Span outs[] = {{dx, rows, hp * 2, dx_stride * 2}, {dB, rows, gn * 2, db_stride * 2},
                         {dC, rows, gn * 2, dc_stride * 2}, whole(ddt, rows * num_heads * 4),
                         whole(dA, num_heads * 4LL), whole(dD, num_heads * 4LL), whole(ddt_bias, num_heads * 4LL),
                         whole(dinitial_state, st * 4), whole(workspace, static_cast<int64_t>(need))};
    const Span ins[] = {{x, rows, hp * 2, x_stride * 2}, {dout, rows, hp * 2, dout_stride * 2},
                        {B, rows, gn * 2, b_stride * 2}, {C, rows, gn * 2, c_stride * 2},
                        whole(dt, rows * num_heads * 4), whole(A, num_heads * 4LL), whole(D, num_heads * 4LL),
                        whole(dt_bias, num_heads * 4LL), whole(initial_state, st * size_of(initial_dtype)),
                        whole(dfinal_state, st * 4), offsets(s)};
    if (any_overlap(outs, ins)) return KDA_ERR_OVERLAP;
    KDA_TRY(check_device());
    kda::ScanParams p;
    scan_params(a, s, rows, &p);
    p.h0 = initial_state;
    p.h0_fp32 = initial_dtype == KDA_DTYPE_FP32;
    p.dout = static_cast<const uint16_t *>(dout);
    p.dout_stride = dout_stride;
    p.dhT = dfinal_state;
    p.dx = static_cast<uint16_t *>(dx);
    p.dx_stride = dx_stride;
    p.dB = static_cast<uint16_t *>(dB);
    p.dC = static_cast<uint16_t *>(dC);
    p.db_stride = db_stride;
    p.dc_stride = dc_stride;
    p.ddt = ddt;
    p.dA = dA;
    p.dD = dD;
    p.ddt_bias = ddt_bias;
    p.dh0 = dinitial_state;
    p.ws = static_cast<float *>(workspace);
    return done(kda::launch_scan_bwd(p, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_scan_decode(const void *x, int64_t x_stride, const float *dt, const float *A, const void *B,
                           int64_t b_stride, const void *C, int64_t c_stride, const float *D, const float *dt_bias,
                           uint32_t flags, int32_t batch, int32_t num_heads, int32_t num_groups, int32_t head_dim,
                           int32_t state_dim, const void *state_in, void *state_out, kda_dtype state_dtype, void *out,
                           kda_stream_t stream) {
    if (batch < 0) return KDA_ERR_BAD_SHAPE;
    const ScanArgs a = {x, x_stride, dt, A, B, b_stride, C, c_stride, D, dt_bias, flags,
                        num_heads, num_groups, head_dim, state_dim};
    KDA_TRY(scan_args(a, batch));
    if ((state_in || state_out) && !float_or_bf16(state_dtype)) return KDA_ERR_STATE_DTYPE;
    if (batch > 0 && !out) return KDA_ERR_NULL_PTR;
    if (!aligned16(out) || !aligned16(state_in) || !aligned16(state_out)) return KDA_ERR_BAD_ALIGNMENT;
    const int64_t units = static_cast<int64_t>(batch) * num_heads;
    if (units > 0x7fffffffLL) return KDA_ERR_TOO_LARGE;
    const int64_t st = units * state_dim * head_dim * size_of(state_dtype), wx = static_cast<int64_t>(num_heads) * head_dim * 2,
                  wb = static_cast<int64_t>(num_groups) * state_dim * 2;
    if (state_in != state_out && overlap(whole(state_in, st), whole(state_out, st))) return KDA_ERR_STATE_OVERLAP;
    const Span outs[] = {whole(out, batch * wx), whole(state_out, st)};
    const Span ins[] = {{x, batch, wx, x_stride * 2}, {B, batch, wb, b_stride * 2}, {C, batch, wb, c_stride * 2},
                        whole(dt, units * 4), whole(A, num_heads * 4LL), whole(D, num_heads * 4LL),
                        whole(dt_bias, num_heads * 4LL)};
    if (any_overlap(outs, ins) || overlap(outs[0], whole(state_in, st))) return KDA_ERR_OVERLAP;
    if (units == 0) return KDA_OK;
    KDA_TRY(check_device());
    kda::ScanDecodeParams p = {};
    p.batch = batch;
    p.H = num_heads;
    p.G = num_groups;
    p.P = head_dim;
    p.N = state_dim;
    p.x = static_cast<const uint16_t *>(x);
    p.B = static_cast<const uint16_t *>(B);
    p.C = static_cast<const uint16_t *>(C);
    p.x_stride = x_stride;
    p.b_stride = b_stride;
    p.c_stride = c_stride;
    p.dt = dt;
    p.A = A;
    p.D = D;
    p.dt_bias = dt_bias;
    p.softplus = (flags & KDA_FLAG_SCAN_SOFTPLUS) != 0;
    p.state_in = state_in;
    p.state_out = state_out;
    p.state_fp32 = state_dtype == KDA_DTYPE_FP32;
    p.out = static_cast<uint16_t *>(out);
    return done(kda::launch_scan_decode(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
