// Host side of the layers around RMA attention (rma_qk_norm_rope, rma_gdn_*): argument checks,
// state layout, launches.  The C declarations and their documentation are in include/rma.h.
#include <cmath>
#include <new>

#include <nvtx3/nvToolsExt.h>

#include "rma_internal.cuh"

namespace rma {
namespace {

struct Nvtx {
    explicit Nvtx(const char* name) { nvtxRangePushA(name); }
    ~Nvtx() { nvtxRangePop(); }
    Nvtx(const Nvtx&) = delete;
    Nvtx& operator=(const Nvtx&) = delete;
};

constexpr uint64_t kAlign = 256;
constexpr int64_t kMaxTokens = 1 << 24;   // batch * n_tok of one call

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// [p, p + pb) and [q, q + qb) share a byte
bool overlap(const void* p, uint64_t pb, const void* q, uint64_t qb) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + qb && b < a + pb;
}

// bytes from the first element of the first row to the last of the last, `rows` rows of `cols`
// elements of `size` bytes, `stride` elements apart
uint64_t span(int64_t rows, int64_t stride, int64_t cols, int64_t size) {
    return (uint64_t)(((rows - 1) * stride + cols) * size);
}

GdnState* as_gdn(rma_gdn_state* p) { return reinterpret_cast<GdnState*>(p); }
const GdnState* as_gdn(const rma_gdn_state* p) { return reinterpret_cast<const GdnState*>(p); }

bool in_state(const GdnState* s, const void* p, uint64_t bytes) {
    return overlap(p, bytes, s->base, s->lay.total_bytes);
}

int channels(const rma_gdn_config& c) { return (2 * c.n_k_heads + c.n_v_heads) * c.head_dim; }

int check_gdn_config(const rma_gdn_config* c) {
    if (!c) return api_fail(RMA_ERR_INVALID_ARG, "config is NULL");
    if (c->batch < 1 || c->n_layers < 1 || c->n_k_heads < 1 || c->n_v_heads < 1)
        return api_fail(RMA_ERR_INVALID_ARG, "batch, n_layers, n_k_heads and n_v_heads must be >= 1");
    if (c->n_v_heads % c->n_k_heads != 0)
        return api_fail(RMA_ERR_INVALID_ARG, "n_v_heads must be a multiple of n_k_heads");
    if (c->head_dim != kGdnDim || c->conv_width != kConvWidth)
        return api_fail(RMA_ERR_UNSUPPORTED, "the library implements head_dim == 128 and conv_width == 4");
    if (c->qk_l2norm != 0 && c->qk_l2norm != 1) return api_fail(RMA_ERR_INVALID_ARG, "qk_l2norm must be 0 or 1");
    if (!(std::isfinite(c->l2_eps) && c->l2_eps >= 0.f))
        return api_fail(RMA_ERR_INVALID_ARG, "l2_eps must be finite and >= 0");
    // (a key far below a larger eps, times a decay, would leave FP32's normal numbers)
    if (c->l2_eps > 1e30f) return api_fail(RMA_ERR_UNSUPPORTED, "l2_eps > 1e30");
    if (!std::isfinite(c->scale)) return api_fail(RMA_ERR_INVALID_ARG, "scale must be finite");
    if ((int64_t)c->batch * c->n_v_heads > (1 << 22)) return api_fail(RMA_ERR_UNSUPPORTED, "batch * n_v_heads > 2^22");
    if ((2ll * c->n_k_heads + c->n_v_heads) * c->head_dim > (1 << 20))
        return api_fail(RMA_ERR_UNSUPPORTED, "more than 2^20 channels");
    if (c->n_layers > (1 << 16)) return api_fail(RMA_ERR_UNSUPPORTED, "n_layers > 2^16");
    return RMA_OK;
}

void gdn_layout(const rma_gdn_config& c, rma_gdn_layout& L) {
    const uint64_t lb = (uint64_t)c.n_layers * c.batch;
    uint64_t off = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t o = off;
        off = (off + bytes + kAlign - 1) / kAlign * kAlign;
        return o;
    };
    L.conv = take(lb * (kConvWidth - 1) * channels(c) * 2);
    L.delta = take(lb * c.n_v_heads * kGdnDim * kGdnDim * 4);
    L.status = take(4);
    L.total_bytes = off;
}

int check_device(int device) {
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return api_cuda_fail(e, "querying the device");
    if (dev != device)
        return api_fail(RMA_ERR_INVALID_ARG, "the current device is not the one the state was laid out on");
    return RMA_OK;
}

// state, layer and n_tok of a gdn call (no CUDA call yet)
int check_call(const GdnState* s, int layer, int n_tok) {
    if (!s) return api_fail(RMA_ERR_INVALID_ARG, "state is NULL");
    if (layer < 0 || layer >= s->cfg.n_layers) return api_fail(RMA_ERR_INVALID_ARG, "layer index out of range");
    if (n_tok < 1) return api_fail(RMA_ERR_INVALID_ARG, "n_tok must be >= 1");
    if ((int64_t)n_tok * s->cfg.batch > kMaxTokens) return api_fail(RMA_ERR_UNSUPPORTED, "batch * n_tok > 2^24");
    return RMA_OK;
}

int launched(cudaError_t e, const char* what, void* stream) {
    if (e == cudaErrorNotSupported) return api_fail(RMA_ERR_UNSUPPORTED, "the call needs more blocks than a launch can have");
    if (e != cudaSuccess) return api_cuda_fail(e, what);
    api_note_launch(static_cast<cudaStream_t>(stream));
    return RMA_OK;
}

// The arguments the two delta-rule calls share.
int delta_args(const GdnState* s, int layer, int n, const uint16_t* qkv, const uint16_t* a, const uint16_t* b,
               int64_t ab_stride, const float* a_log, const float* dt_bias, const int32_t* lens, uint16_t* out,
               DeltaArgs& d) {
    const rma_gdn_config& c = s->cfg;
    if (!qkv || !a || !b || !a_log || !dt_bias || !out) return api_fail(RMA_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (!aligned(qkv, 16) || !aligned(out, 16)) return api_fail(RMA_ERR_MISALIGNED, "qkv and out need 16-byte alignment");
    if (!aligned(a, 2) || !aligned(b, 2) || !aligned(a_log, 4) || !aligned(dt_bias, 4) || !aligned(lens, 4))
        return api_fail(RMA_ERR_MISALIGNED, "a and b need 2-byte alignment, a_log, dt_bias and lens 4-byte");
    if (ab_stride < c.n_v_heads || ab_stride > (1ll << 32))
        return api_fail(RMA_ERR_INVALID_ARG, "ab_stride must be >= n_v_heads (and <= 2^32)");
    const int64_t rows = (int64_t)c.batch * n;
    const int C = channels(c);
    const uint64_t ob = span(rows, c.n_v_heads * kGdnDim, c.n_v_heads * kGdnDim, 2);
    const uint64_t ab = span(rows, ab_stride, c.n_v_heads, 2);
    const uint64_t xb = span(rows, C, C, 2), hb = 4ull * c.n_v_heads;
    if (in_state(s, qkv, xb) || in_state(s, a, ab) || in_state(s, b, ab) || in_state(s, a_log, hb) ||
        in_state(s, dt_bias, hb) || in_state(s, lens, 4ull * c.batch))
        return api_fail(RMA_ERR_INVALID_ARG, "an input overlaps the state");
    if (overlap(out, ob, qkv, xb) || overlap(out, ob, a, ab) || overlap(out, ob, b, ab) ||
        overlap(out, ob, a_log, hb) || overlap(out, ob, dt_bias, hb) || overlap(out, ob, lens, 4ull * c.batch) ||
        in_state(s, out, ob))
        return api_fail(RMA_ERR_INVALID_ARG, "out overlaps an input or the state");
    const uint64_t l = (uint64_t)layer;
    d.qkv = qkv;
    d.a = a;
    d.b = b;
    d.ab_stride = ab_stride;
    d.a_log = a_log;
    d.dt_bias = dt_bias;
    d.lens = lens;
    d.state = reinterpret_cast<float*>(s->base + s->lay.delta) + l * c.batch * c.n_v_heads * kGdnDim * kGdnDim;
    d.out = out;
    d.ws = nullptr;
    d.status = reinterpret_cast<uint32_t*>(s->base + s->lay.status);
    d.B = c.batch;
    d.n = n;
    d.HK = c.n_k_heads;
    d.HV = c.n_v_heads;
    d.C = C;
    d.l2norm = c.qk_l2norm;
    d.l2_eps = c.l2_eps;
    d.scale = c.scale;
    d.sm_count = s->sm_count;
    return RMA_OK;
}

}  // namespace
}  // namespace rma

using namespace rma;

extern "C" {

int rma_qk_norm_rope(rma_state* st, int layer, int n_tok, const uint16_t* q, int64_t q_stride, const uint16_t* k,
                     int64_t k_stride, const float* w_q, const float* w_k, float eps, const double* inv_freq,
                     int rotary_dim, int interleaved, const int32_t* positions, uint16_t* q_out, uint16_t* k_out,
                     void* stream) {
    Nvtx range("rma_qk_norm_rope");
    const State* s = reinterpret_cast<const State*>(st);
    if (!s) return api_fail(RMA_ERR_INVALID_ARG, "state is NULL");
    const rma_config& c = s->cfg;
    if (layer < 0 || layer >= c.n_layers) return api_fail(RMA_ERR_INVALID_ARG, "layer index out of range");
    if (n_tok < 1) return api_fail(RMA_ERR_INVALID_ARG, "n_tok must be >= 1");
    if (rotary_dim < 0 || rotary_dim > kHeadDim || rotary_dim % 2 != 0)
        return api_fail(RMA_ERR_INVALID_ARG, "rotary_dim must be even, 0 to 256");
    if (interleaved != 0 && interleaved != 1) return api_fail(RMA_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    if (!(std::isfinite(eps) && eps >= 0.f)) return api_fail(RMA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!q || !k || !w_q || !w_k || !q_out || !k_out || (rotary_dim > 0 && !inv_freq))
        return api_fail(RMA_ERR_INVALID_ARG, "a tensor pointer is NULL");
    const int64_t rows = (int64_t)c.batch * n_tok, kr = (int64_t)c.n_groups * kHeadDim, qr = kr * kQPerGroup;
    if (rows > kMaxTokens || rows * c.n_groups > 0x7fffffffll)
        return api_fail(RMA_ERR_UNSUPPORTED, "batch * n_tok > 2^24, or times n_groups > 2^31 - 1");
    if (q_stride < qr || k_stride < kr || q_stride % 8 != 0 || k_stride % 8 != 0 || q_stride > (1ll << 32) ||
        k_stride > (1ll << 32))
        return api_fail(RMA_ERR_INVALID_ARG, "q_stride and k_stride must be multiples of 8, at least a row (and <= 2^32)");
    const void* a16[] = {q, k, w_q, w_k, q_out, k_out};
    for (const void* p : a16)
        if (!aligned(p, 16)) return api_fail(RMA_ERR_MISALIGNED, "q, k, w_q, w_k, q_out, k_out need 16-byte alignment");
    if (!aligned(inv_freq, 8) || !aligned(positions, 4))
        return api_fail(RMA_ERR_MISALIGNED, "inv_freq needs 8-byte alignment, positions 4-byte");
    const uint64_t qb = span(rows, q_stride, qr, 2), kb = span(rows, k_stride, kr, 2);
    const uint64_t qo = span(rows, qr, qr, 2), ko = span(rows, kr, kr, 2);
    struct Range {
        const void* p;
        uint64_t bytes;
    };
    const Range in[] = {{q, qb}, {k, kb}, {w_q, kHeadDim * 4}, {w_k, kHeadDim * 4},
                        {inv_freq, (uint64_t)rotary_dim * 4}, {positions, (uint64_t)rows * 4}, {s->base, s->lay.total_bytes}};
    bool bad = overlap(q_out, qo, k_out, ko);
    for (const Range& r : in) {
        if (r.bytes == 0) continue;
        if (!(r.p == q && q_out == q && q_stride == qr) && overlap(q_out, qo, r.p, r.bytes)) bad = true;
        if (!(r.p == k && k_out == k && k_stride == kr) && overlap(k_out, ko, r.p, r.bytes)) bad = true;
    }
    if (bad) return api_fail(RMA_ERR_INVALID_ARG, "q_out or k_out overlaps an input, the state or the other (other than in place)");
    const int rc = check_device(s->device);
    if (rc != RMA_OK) return rc;
    RopeArgs a;
    a.q = q;
    a.k = k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.w_q = w_q;
    a.w_k = w_k;
    a.inv_freq = inv_freq;
    a.positions = positions;
    a.counters = reinterpret_cast<const int32_t*>(s->base + s->lay.counters) + (uint64_t)layer * c.batch * c.n_groups * 4;
    a.status = reinterpret_cast<uint32_t*>(s->base + s->lay.status);
    a.q_out = q_out;
    a.k_out = k_out;
    a.B = c.batch;
    a.n = n_tok;
    a.G = c.n_groups;
    a.half = rotary_dim / 2;
    a.interleaved = interleaved;
    a.eps = eps;
    return launched(launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)), "launching rma_qk_norm_rope", stream);
}

size_t rma_gdn_state_bytes(const rma_gdn_config* cfg) {
    if (check_gdn_config(cfg) != RMA_OK) return 0;
    rma_gdn_layout L;
    gdn_layout(*cfg, L);
    return (size_t)L.total_bytes;
}

int rma_gdn_state_alloc(const rma_gdn_config* cfg, void* dev_buf, size_t dev_bytes, void* stream, rma_gdn_state** out) {
    const int rc = check_gdn_config(cfg);
    if (rc != RMA_OK) return rc;
    if (!dev_buf || !out) return api_fail(RMA_ERR_INVALID_ARG, "dev_buf and out must be non-NULL");
    if (!aligned(dev_buf, kAlign)) return api_fail(RMA_ERR_MISALIGNED, "dev_buf must be 256-byte aligned");
    rma_gdn_layout L;
    gdn_layout(*cfg, L);
    if (dev_bytes < L.total_bytes)
        return api_fail(RMA_ERR_BUFFER_TOO_SMALL, "state buffer smaller than rma_gdn_state_bytes()");
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return api_cuda_fail(e, "querying the device");
    GdnState* s = new (std::nothrow) GdnState;
    if (!s) return api_fail(RMA_ERR_INVALID_ARG, "host allocation of the handle failed");
    s->cfg = *cfg;
    s->lay = L;
    s->base = static_cast<uint8_t*>(dev_buf);
    s->sm_count = sms;
    s->device = dev;
    e = cudaMemsetAsync(s->base, 0, L.total_bytes, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        delete s;
        return api_cuda_fail(e, "zeroing the state");
    }
    *out = reinterpret_cast<rma_gdn_state*>(s);
    return RMA_OK;
}

int rma_gdn_state_layout(const rma_gdn_state* st, rma_gdn_layout* out) {
    if (!st || !out) return api_fail(RMA_ERR_INVALID_ARG, "state and out must be non-NULL");
    *out = as_gdn(st)->lay;
    return RMA_OK;
}

void rma_gdn_state_free(rma_gdn_state* st) { delete as_gdn(st); }

int rma_gdn_workspace_bytes(const rma_gdn_state* st, int n_tok, size_t* out) {
    if (!st || !out) return api_fail(RMA_ERR_INVALID_ARG, "state and out must be non-NULL");
    const int rc = check_call(as_gdn(st), 0, n_tok);
    if (rc != RMA_OK) return rc;
    *out = gdn_prefill_workspace_bytes(as_gdn(st)->cfg, n_tok);
    return RMA_OK;
}

int rma_gdn_conv(rma_gdn_state* st, int layer, int n_tok, const uint16_t* x, int64_t x_stride, const float* w,
                 const float* bias, const int32_t* lens, uint16_t* out, void* stream) {
    Nvtx range("rma_gdn_conv");
    const GdnState* s = as_gdn(st);
    int rc = check_call(s, layer, n_tok);
    if (rc != RMA_OK) return rc;
    const rma_gdn_config& c = s->cfg;
    const int C = channels(c);
    if (!x || !w || !out) return api_fail(RMA_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(out, 16))
        return api_fail(RMA_ERR_MISALIGNED, "x, w, bias and out need 16-byte alignment");
    if (!aligned(lens, 4)) return api_fail(RMA_ERR_MISALIGNED, "lens needs 4-byte alignment");
    if (x_stride < C || x_stride % 8 != 0 || x_stride > (1ll << 32))
        return api_fail(RMA_ERR_INVALID_ARG, "x_stride must be a multiple of 8, at least the channels (and <= 2^32)");
    const int64_t rows = (int64_t)c.batch * n_tok;
    const uint64_t ob = span(rows, C, C, 2), xb = span(rows, x_stride, C, 2);
    if (in_state(s, x, xb) || in_state(s, w, 16ull * C) || in_state(s, bias, 4ull * C) || in_state(s, lens, 4ull * c.batch))
        return api_fail(RMA_ERR_INVALID_ARG, "an input overlaps the state");
    if (overlap(out, ob, x, xb) || overlap(out, ob, w, 16ull * C) ||
        overlap(out, ob, bias, 4ull * C) || overlap(out, ob, lens, 4ull * c.batch) || in_state(s, out, ob))
        return api_fail(RMA_ERR_INVALID_ARG, "out overlaps an input or the state");
    rc = check_device(s->device);
    if (rc != RMA_OK) return rc;
    ConvArgs a;
    a.x = x;
    a.x_stride = x_stride;
    a.w = w;
    a.bias = bias;
    a.lens = lens;
    a.state = reinterpret_cast<uint16_t*>(s->base + s->lay.conv) + (uint64_t)layer * c.batch * (kConvWidth - 1) * C;
    a.out = out;
    a.status = reinterpret_cast<uint32_t*>(s->base + s->lay.status);
    a.B = c.batch;
    a.n = n_tok;
    a.C = C;
    return launched(launch_gdn_conv(a, static_cast<cudaStream_t>(stream)), "launching rma_gdn_conv", stream);
}

int rma_gdn_decode_step(rma_gdn_state* st, int layer, const uint16_t* qkv, const uint16_t* a, const uint16_t* b,
                        int64_t ab_stride, const float* a_log, const float* dt_bias, uint16_t* out, void* stream) {
    Nvtx range("rma_gdn_decode_step");
    const GdnState* s = as_gdn(st);
    int rc = check_call(s, layer, 1);
    if (rc != RMA_OK) return rc;
    DeltaArgs d;
    rc = delta_args(s, layer, 1, qkv, a, b, ab_stride, a_log, dt_bias, nullptr, out, d);
    if (rc == RMA_OK) rc = check_device(s->device);
    if (rc != RMA_OK) return rc;
    return launched(launch_gdn_recurrent(d, static_cast<cudaStream_t>(stream)), "launching rma_gdn_decode_step", stream);
}

int rma_gdn_prefill(rma_gdn_state* st, int layer, int n_tok, const uint16_t* qkv, const uint16_t* a,
                    const uint16_t* b, int64_t ab_stride, const float* a_log, const float* dt_bias,
                    const int32_t* lens, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
    Nvtx range("rma_gdn_prefill");
    const GdnState* s = as_gdn(st);
    int rc = check_call(s, layer, n_tok);
    if (rc != RMA_OK) return rc;
    DeltaArgs d;
    rc = delta_args(s, layer, n_tok, qkv, a, b, ab_stride, a_log, dt_bias, lens, out, d);
    if (rc != RMA_OK) return rc;
    size_t need = 0;
    rc = rma_gdn_workspace_bytes(st, n_tok, &need);
    if (rc != RMA_OK) return rc;
    if (!ws) return api_fail(RMA_ERR_INVALID_ARG, "ws is NULL");
    if (!aligned(ws, kAlign)) return api_fail(RMA_ERR_MISALIGNED, "ws must be 256-byte aligned");
    if (ws_bytes < need) return api_fail(RMA_ERR_BUFFER_TOO_SMALL, "workspace smaller than rma_gdn_workspace_bytes(st, n_tok)");
    const int64_t rows = (int64_t)s->cfg.batch * n_tok;
    const uint64_t ab = span(rows, ab_stride, s->cfg.n_v_heads, 2);
    if (overlap(ws, need, qkv, span(rows, d.C, d.C, 2)) || overlap(ws, need, a, ab) || overlap(ws, need, b, ab) ||
        overlap(ws, need, a_log, 4ull * d.HV) || overlap(ws, need, dt_bias, 4ull * d.HV) ||
        overlap(ws, need, lens, 4ull * d.B) || overlap(ws, need, out, span(rows, d.HV * kGdnDim, d.HV * kGdnDim, 2)) ||
        in_state(s, ws, need))
        return api_fail(RMA_ERR_INVALID_ARG, "ws overlaps a tensor of the call or the state");
    rc = check_device(s->device);
    if (rc != RMA_OK) return rc;
    d.ws = static_cast<uint8_t*>(ws);
    return launched(launch_gdn_prefill(d, static_cast<cudaStream_t>(stream)), "launching rma_gdn_prefill", stream);
}

int rma_gdn_get_status(rma_gdn_state* st, void* stream, uint32_t* flags) {
    if (!st || !flags) return api_fail(RMA_ERR_INVALID_ARG, "state and flags must be non-NULL");
    const GdnState* s = as_gdn(st);
    const int rc = check_device(s->device);
    if (rc != RMA_OK) return rc;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    uint32_t h = 0;
    cudaError_t e = cudaMemcpyAsync(&h, s->base + s->lay.status, 4, cudaMemcpyDeviceToHost, cs);
    if (e == cudaSuccess) e = cudaMemsetAsync(s->base + s->lay.status, 0, 4, cs);
    if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
    if (e != cudaSuccess) return api_cuda_fail(e, "reading the status word");
    *flags = h;
    return RMA_OK;
}

}  // extern "C"
