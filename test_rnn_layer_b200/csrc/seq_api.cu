// C ABI of the sequence operators beside the layer (rotary positions, window
// attention, gated linear recurrence): argument checks and launches.
#include <algorithm>
#include <climits>
#include <cmath>

#include "../../include/tttmlp.h"
#include "internal.h"

using namespace ttt;

namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxRows = 1 << 30;
constexpr int kMaxWindowRows = 1 << 28;   // positions plus a window of any width stay inside an int
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

#define SEQ_TRY(expr)                                                                                       \
    do {                                                                                                    \
        cudaError_t e_ = (expr);                                                                            \
        if (e_ != cudaSuccess) return set_error(TTT_ERR_CUDA, "%s: %s", #expr, cudaGetErrorString(e_));     \
    } while (0)

bool aligned(const void* p, size_t n = 16) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

ttt_status need(const void* p, const char* name) {
    if (!p) return set_error(TTT_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p)) return set_error(TTT_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
    return TTT_OK;
}

ttt_status need_rows(const void* p, int ld, long long cols, const char* name) {
    const ttt_status st = need(p, name);
    if (st != TTT_OK) return st;
    if (ld < cols || ld % 8) return set_error(TTT_ERR_INVALID_ARG, "%s: row stride %d must be a multiple of 8, at least %lld", name, ld, cols);
    return TTT_OK;
}

#define SEQ_NEED(call)                       \
    do {                                     \
        const ttt_status st_ = (call);       \
        if (st_ != TTT_OK) return st_;       \
    } while (0)

ttt_status check_workspace(const void* ws, size_t bytes, size_t want) {
    if (!ws || !aligned(ws, kAlign)) return set_error(TTT_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
    if (bytes < want) return set_error(TTT_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", bytes, want);
    return TTT_OK;
}

// Whether two row arrays share memory (byte ranges from the first row's start to the last row's end).
bool overlap(const void* a, long long rows_a, long long ld_a, long long cols_a, size_t ea, const void* b,
             long long rows_b, long long ld_b, long long cols_b, size_t eb) {
    if (!a || !b || rows_a < 1 || rows_b < 1) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    const uintptr_t a1 = a0 + ((rows_a - 1) * ld_a + cols_a) * ea, b1 = b0 + ((rows_b - 1) * ld_b + cols_b) * eb;
    if (a0 >= b1 || b0 >= a1) return false;
    // columns side by side in rows of the same stride do not meet
    if (ld_a * ea == ld_b * eb) {
        const uintptr_t pitch = ld_a * ea, off = (b0 > a0 ? b0 - a0 : a0 - b0) % pitch;
        const uintptr_t low = b0 > a0 ? cols_a * ea : cols_b * eb, high = b0 > a0 ? cols_b * eb : cols_a * ea;
        if (off >= low && off + high <= pitch) return false;
    }
    return true;
}

ttt_status check_sequences(int n_seq, const int* cu) {
    if (n_seq < 1 || n_seq > kMaxRows) return set_error(TTT_ERR_INVALID_ARG, "n_seq=%d must be at least 1", n_seq);
    if (!cu && n_seq != 1) return set_error(TTT_ERR_INVALID_ARG, "n_seq=%d needs the sequences' offsets", n_seq);
    if (cu && !aligned(cu, 4)) return set_error(TTT_ERR_INVALID_ARG, "sequence offsets are not 4-byte aligned");
    return TTT_OK;
}

// ---------------------------------------------------------------- window attention
ttt_status check_window(const ttt_window_desc* q) {
    if (!q) return set_error(TTT_ERR_INVALID_ARG, "desc is NULL");
    if (q->Tq < 0 || q->Tk < 0 || q->Tq > kMaxWindowRows || q->Tk > kMaxWindowRows)
        return set_error(TTT_ERR_INVALID_ARG, "Tq=%d, Tk=%d must lie in [0, 2^28]", q->Tq, q->Tk);
    if (q->Hq < 1 || q->Hk < 1 || q->Hq % q->Hk || q->Hq > 65535)
        return set_error(TTT_ERR_INVALID_ARG, "Hq=%d must be a multiple of Hk=%d, both at least 1", q->Hq, q->Hk);
    if (q->d != 64) return set_error(TTT_ERR_UNSUPPORTED, "head dim %d: the window attention has 64", q->d);
    if (q->left < 0 || q->right < 0 || q->sinks < 0)
        return set_error(TTT_ERR_INVALID_ARG, "left=%d, right=%d, sinks=%d must not be negative", q->left, q->right, q->sinks);
    if (!(q->scale > 0.f) || !std::isfinite(q->scale))
        return set_error(TTT_ERR_INVALID_ARG, "scale must be positive and finite");
    if (q->n_seq < 1 || q->n_seq > kMaxRows) return set_error(TTT_ERR_INVALID_ARG, "n_seq=%d must be at least 1", q->n_seq);
    // blocks of 128 rows and heads are counted in an int (with room for the sinks' chunks and the counter's overshoot)
    if (std::max((q->Tq / 128LL + q->n_seq) * q->Hq, (q->Tk / 128LL + q->n_seq) * q->Hk) > (1LL << 31) - (1 << 21))
        return set_error(TTT_ERR_UNSUPPORTED, "n_seq=%d, Hq=%d: too many blocks of rows for one call", q->n_seq, q->Hq);
    return TTT_OK;
}

ttt_status fill_window(WindowArgs& a, const ttt_window_desc& q, const int* cu_q, const int* cu_k, const void* Q,
                       int ld_q, const void* K, int ld_k, const void* V, int ld_v) {
    if ((cu_q == nullptr) != (cu_k == nullptr))
        return set_error(TTT_ERR_INVALID_ARG, "cu_q and cu_k are given both or not at all");
    SEQ_NEED(check_sequences(q.n_seq, cu_q));
    SEQ_NEED(check_sequences(q.n_seq, cu_k));
    if (q.Tq) SEQ_NEED(need_rows(Q, ld_q, (long long)q.Hq * q.d, "Q"));
    if (q.Tk) {
        SEQ_NEED(need_rows(K, ld_k, (long long)q.Hk * q.d, "K"));
        SEQ_NEED(need_rows(V, ld_v, (long long)q.Hk * q.d, "V"));
    }
    a.Tq = q.Tq; a.Tk = q.Tk; a.n_seq = q.n_seq; a.Hq = q.Hq; a.Hk = q.Hk;
    // a side that reaches past every key is the same as one that ends there; cut, p +- side stays in an int
    a.left = std::min(q.left, q.Tq + q.Tk);
    a.right = std::min(q.right, q.Tq + q.Tk);
    a.sinks = std::min(q.sinks, q.Tk);
    a.scale = q.scale;
    a.cu_q = cu_q; a.cu_k = cu_k;
    a.Q = static_cast<const __nv_bfloat16*>(Q); a.ld_q = ld_q;
    a.K = static_cast<const __nv_bfloat16*>(K); a.ld_k = ld_k;
    a.V = static_cast<const __nv_bfloat16*>(V); a.ld_v = ld_v;
    return TTT_OK;
}

}  // namespace

// ---------------------------------------------------------------- rotary positions
extern "C" TTT_API ttt_status ttt_rope(const ttt_rope_desc* desc, const void* X, int ld_x, void* Y, int ld_y,
                               const int* positions, int pos0, int inverse, ttt_stream_t stream) {
    if (!desc) return set_error(TTT_ERR_INVALID_ARG, "desc is NULL");
    const ttt_rope_desc& q = *desc;
    if (q.T < 0 || q.T > kMaxRows || q.H < 1) return set_error(TTT_ERR_INVALID_ARG, "T=%d, H=%d", q.T, q.H);
    if (q.d < 8 || q.d % 8) return set_error(TTT_ERR_INVALID_ARG, "d=%d must be a multiple of 8", q.d);
    if (q.d > 2 * kRopeMaxPairs) return set_error(TTT_ERR_UNSUPPORTED, "d=%d above %d", q.d, 2 * kRopeMaxPairs);
    if (q.rot < 2 || q.rot % 2 || q.rot > q.d) return set_error(TTT_ERR_INVALID_ARG, "rot=%d must be even, 2 to d=%d", q.rot, q.d);
    if (q.layout != TTT_ROPE_HALF && q.layout != TTT_ROPE_INTERLEAVED) return set_error(TTT_ERR_INVALID_ARG, "layout %d", (int)q.layout);
    if (q.x_dtype != TTT_F32 && q.x_dtype != TTT_BF16) return set_error(TTT_ERR_INVALID_ARG, "x_dtype %d", (int)q.x_dtype);
    if (!(q.base > 1.0) || !std::isfinite(q.base)) return set_error(TTT_ERR_INVALID_ARG, "base must be finite and above 1");
    if (!std::isfinite(q.amplitude)) return set_error(TTT_ERR_INVALID_ARG, "amplitude must be finite");
    if (q.scaling < TTT_ROPE_SCALE_NONE || q.scaling > TTT_ROPE_SCALE_RAMP) return set_error(TTT_ERR_INVALID_ARG, "scaling %d", (int)q.scaling);
    if (q.scaling != TTT_ROPE_SCALE_NONE && (!(q.factor >= 1.0) || !std::isfinite(q.factor)))
        return set_error(TTT_ERR_INVALID_ARG, "factor must be finite and at least 1");
    if (q.scaling == TTT_ROPE_SCALE_BASE && q.rot < 4) return set_error(TTT_ERR_INVALID_ARG, "a scaled base needs rot above 2");
    if (q.scaling == TTT_ROPE_SCALE_RAMP &&
        (!(q.length > 0.0) || !std::isfinite(q.length) || !(q.low >= 0.0) || !(q.high > q.low) || !std::isfinite(q.high)))
        return set_error(TTT_ERR_INVALID_ARG, "the ramp needs length > 0 and 0 <= low < high");
    if (q.T == 0) return TTT_OK;
    SEQ_NEED(need_rows(X, ld_x, (long long)q.H * q.d, "X"));
    SEQ_NEED(need_rows(Y, ld_y, (long long)q.H * q.d, "Y"));
    if (positions && !aligned(positions, 4)) return set_error(TTT_ERR_INVALID_ARG, "positions are not 4-byte aligned");
    const size_t e = q.x_dtype == TTT_BF16 ? 2 : 4;
    if (!(X == Y && ld_x == ld_y) && overlap(X, q.T, ld_x, (long long)q.H * q.d, e, Y, q.T, ld_y, (long long)q.H * q.d, e))
        return set_error(TTT_ERR_INVALID_ARG, "Y overlaps X and is not X itself");
    RopeArgs a{};
    a.X = X; a.Y = Y; a.ld_x = ld_x; a.ld_y = ld_y;
    a.positions = positions; a.pos0 = pos0;
    a.T = q.T; a.H = q.H; a.d = q.d; a.rot = q.rot; a.half = q.layout == TTT_ROPE_HALF; a.bf16 = q.x_dtype == TTT_BF16;
    a.inverse = inverse != 0;
    a.amplitude = (float)q.amplitude;
    const double two_pi = 6.283185307179586476925286766559;
    const double base = q.scaling == TTT_ROPE_SCALE_BASE ? q.base * std::pow(q.factor, (double)q.rot / (q.rot - 2)) : q.base;
    for (int i = 0; i < q.rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / q.rot);
        if (q.scaling == TTT_ROPE_SCALE_LINEAR) f /= q.factor;
        if (q.scaling == TTT_ROPE_SCALE_RAMP) {
            const double r = q.length * f / two_pi;
            const double keep = std::min(1.0, std::max(0.0, (r - q.low) / (q.high - q.low)));
            f *= keep + (1.0 - keep) / q.factor;
        }
        a.turns[i] = f / two_pi;
    }
    SEQ_TRY(launch_rope(a, reinterpret_cast<cudaStream_t>(stream)));
    return TTT_OK;
}

// ---------------------------------------------------------------- window attention
extern "C" TTT_API size_t ttt_window_attention_workspace_size(const ttt_window_desc* desc) {
    return check_window(desc) == TTT_OK ? kAlign : 0;
}

extern "C" TTT_API size_t ttt_window_attention_backward_workspace_size(const ttt_window_desc* desc) {
    if (check_window(desc) != TTT_OK) return 0;
    WindowArgs a{};
    a.Tq = desc->Tq; a.n_seq = desc->n_seq; a.Hq = desc->Hq; a.Hk = desc->Hk;
    return kAlign + align_up((size_t)desc->Hq * desc->Tq * sizeof(float)) + align_up((size_t)desc->Hk * desc->Tk) +
           (size_t)window_partial_floats(a) * sizeof(float);
}

extern "C" TTT_API ttt_status ttt_window_attention(const ttt_window_desc* desc, const int* cu_q, const int* cu_k, const void* Q,
                                           int ld_q, const void* K, int ld_k, const void* V, int ld_v,
                                           const void* Xres, void* Out, int ld_out, float* Lse, void* workspace,
                                           size_t workspace_bytes, ttt_stream_t stream) {
    SEQ_NEED(check_window(desc));
    const ttt_window_desc& q = *desc;
    WindowArgs a{};
    SEQ_NEED(fill_window(a, q, cu_q, cu_k, Q, ld_q, K, ld_k, V, ld_v));
    SEQ_NEED(check_workspace(workspace, workspace_bytes, kAlign));
    const long long wq = (long long)q.Hq * q.d, wk = (long long)q.Hk * q.d;
    if (q.Tq) SEQ_NEED(need_rows(Out, ld_out, wq, "Out"));
    if (Xres) SEQ_NEED(need(Xres, "Xres"));
    if (Lse && !aligned(Lse)) return set_error(TTT_ERR_INVALID_ARG, "Lse is not 16-byte aligned");
    if (overlap(Out, q.Tq, ld_out, wq, 2, Q, q.Tq, ld_q, wq, 2) || overlap(Out, q.Tq, ld_out, wq, 2, K, q.Tk, ld_k, wk, 2) ||
        overlap(Out, q.Tq, ld_out, wq, 2, V, q.Tk, ld_v, wk, 2))
        return set_error(TTT_ERR_INVALID_ARG, "Out overlaps Q, K or V");
    if (Xres != Out && overlap(Out, q.Tq, ld_out, wq, 2, Xres, q.Tq, ld_out, wq, 2))
        return set_error(TTT_ERR_INVALID_ARG, "Xres overlaps Out and is not Out itself");
    a.Xres = static_cast<const __nv_bfloat16*>(Xres);
    a.Out = static_cast<__nv_bfloat16*>(Out);
    a.ld_out = ld_out;
    a.Lse = Lse;
    a.status = static_cast<int*>(workspace);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    SEQ_TRY(cudaMemsetAsync(workspace, 0, 16, s));
    if (q.Tq) SEQ_TRY(launch_window_attention(a, s));
    return TTT_OK;
}

extern "C" TTT_API ttt_status ttt_window_attention_backward(const ttt_window_desc* desc, const int* cu_q, const int* cu_k,
                                                    const void* Q, int ld_q, const void* K, int ld_k, const void* V,
                                                    int ld_v, const void* Out, int ld_out, const float* Lse,
                                                    const void* dOut, int ld_do, void* dQ, int ld_dq, void* dK,
                                                    int ld_dk, void* dV, int ld_dv, void* workspace,
                                                    size_t workspace_bytes, ttt_stream_t stream) {
    SEQ_NEED(check_window(desc));
    const ttt_window_desc& q = *desc;
    WindowArgs a{};
    SEQ_NEED(fill_window(a, q, cu_q, cu_k, Q, ld_q, K, ld_k, V, ld_v));
    SEQ_NEED(check_workspace(workspace, workspace_bytes, ttt_window_attention_backward_workspace_size(desc)));
    const long long wq = (long long)q.Hq * q.d, wk = (long long)q.Hk * q.d;
    if (q.Tq) {
        SEQ_NEED(need_rows(Out, ld_out, wq, "Out"));
        SEQ_NEED(need_rows(dOut, ld_do, wq, "dOut"));
        SEQ_NEED(need_rows(dQ, ld_dq, wq, "dQ"));
        SEQ_NEED(need(Lse, "Lse"));
    }
    if (q.Tk) {
        SEQ_NEED(need_rows(dK, ld_dk, wk, "dK"));
        SEQ_NEED(need_rows(dV, ld_dv, wk, "dV"));
    }
    struct Rows { const void* p; long long rows, ld, cols; };
    const Rows in[] = {{Q, q.Tq, ld_q, wq}, {Out, q.Tq, ld_out, wq}, {dOut, q.Tq, ld_do, wq}, {K, q.Tk, ld_k, wk}, {V, q.Tk, ld_v, wk}};
    const Rows out[] = {{dQ, q.Tq, ld_dq, wq}, {dK, q.Tk, ld_dk, wk}, {dV, q.Tk, ld_dv, wk}};
    for (int i = 0; i < 3; ++i) {
        for (const Rows& r : in)
            if (overlap(out[i].p, out[i].rows, out[i].ld, out[i].cols, 2, r.p, r.rows, r.ld, r.cols, 2))
                return set_error(TTT_ERR_INVALID_ARG, "a gradient overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].rows, out[i].ld, out[i].cols, 2, out[j].p, out[j].rows, out[j].ld, out[j].cols, 2))
                return set_error(TTT_ERR_INVALID_ARG, "two gradients overlap");
    }
    a.Out = static_cast<__nv_bfloat16*>(const_cast<void*>(Out));
    a.ld_out = ld_out;
    a.Lse = const_cast<float*>(Lse);
    a.dOut = static_cast<const __nv_bfloat16*>(dOut); a.ld_do = ld_do;
    a.dQ = static_cast<__nv_bfloat16*>(dQ); a.ld_dq = ld_dq;
    a.dK = static_cast<__nv_bfloat16*>(dK); a.ld_dk = ld_dk;
    a.dV = static_cast<__nv_bfloat16*>(dV); a.ld_dv = ld_dv;
    a.status = static_cast<int*>(workspace);
    a.grad_scale = a.left == 0 && a.right == 0 && a.sinks == 0 ? 0.f : a.scale;
    char* space = static_cast<char*>(workspace) + kAlign;
    a.delta = reinterpret_cast<float*>(space);
    space += align_up((size_t)q.Hq * q.Tq * sizeof(float));
    a.key_odd = reinterpret_cast<uint8_t*>(space);
    a.partial = reinterpret_cast<float*>(space + align_up((size_t)q.Hk * q.Tk));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    SEQ_TRY(cudaMemsetAsync(workspace, 0, 16, s));
    if (q.Tq || q.Tk) SEQ_TRY(launch_window_attention_backward(a, s));
    return TTT_OK;
}

static ttt_status check_decode(const ttt_window_decode_desc* q) {
    if (!q) return set_error(TTT_ERR_INVALID_ARG, "desc is NULL");
    if (q->B < 0 || q->B > kMaxRows) return set_error(TTT_ERR_INVALID_ARG, "B=%d", q->B);
    if (q->Hq < 1 || q->Hk < 1 || q->Hq % q->Hk || q->Hk > 65535)
        return set_error(TTT_ERR_INVALID_ARG, "Hq=%d must be a multiple of Hk=%d, both at least 1", q->Hq, q->Hk);
    if (q->d != 64) return set_error(TTT_ERR_UNSUPPORTED, "head dim %d: the window attention has 64", q->d);
    if (q->left < 0 || q->sinks < 0 || q->slots < 1 || q->slots > kMaxRows)
        return set_error(TTT_ERR_INVALID_ARG, "slots=%d must be at least 1, left=%d and sinks=%d not negative", q->slots, q->left, q->sinks);
    if (!(q->scale > 0.f) || !std::isfinite(q->scale)) return set_error(TTT_ERR_INVALID_ARG, "scale must be positive and finite");
    if (q->ld_request % 8 || q->ld_slot % 8 || q->ld_head % 8 || q->ld_request < 0 || q->ld_slot < 64 || q->ld_head < 0)
        return set_error(TTT_ERR_INVALID_ARG, "cache strides must be multiples of 8, a slot's at least 64");
    return TTT_OK;
}

extern "C" TTT_API size_t ttt_window_attention_decode_workspace_size(const ttt_window_decode_desc* desc) {
    return check_decode(desc) == TTT_OK ? kAlign : 0;
}

extern "C" TTT_API ttt_status ttt_window_attention_decode(const ttt_window_decode_desc* desc, const void* Q, int ld_q,
                                                  const void* K_new, const void* V_new, int ld_new, void* K_cache,
                                                  void* V_cache, const int* lens, void* Out, int ld_out,
                                                  void* workspace, size_t workspace_bytes, ttt_stream_t stream) {
    SEQ_NEED(check_decode(desc));
    const ttt_window_decode_desc& q = *desc;
    SEQ_NEED(check_workspace(workspace, workspace_bytes, kAlign));
    if (q.B == 0) return TTT_OK;
    SEQ_NEED(need_rows(Q, ld_q, (long long)q.Hq * q.d, "Q"));
    SEQ_NEED(need_rows(Out, ld_out, (long long)q.Hq * q.d, "Out"));
    SEQ_NEED(need(K_cache, "K_cache"));
    SEQ_NEED(need(V_cache, "V_cache"));
    if (!lens || !aligned(lens, 4)) return set_error(TTT_ERR_INVALID_ARG, "lens must be non-NULL and 4-byte aligned");
    if ((K_new == nullptr) != (V_new == nullptr)) return set_error(TTT_ERR_INVALID_ARG, "K_new and V_new are given both or not at all");
    if (K_new) {
        SEQ_NEED(need_rows(K_new, ld_new, (long long)q.Hk * q.d, "K_new"));
        SEQ_NEED(need_rows(V_new, ld_new, (long long)q.Hk * q.d, "V_new"));
    }
    const long long wq = (long long)q.Hq * q.d, wk = (long long)q.Hk * q.d;
    if (overlap(Out, q.B, ld_out, wq, 2, Q, q.B, ld_q, wq, 2) || overlap(Out, q.B, ld_out, wq, 2, K_new, q.B, ld_new, wk, 2) ||
        overlap(Out, q.B, ld_out, wq, 2, V_new, q.B, ld_new, wk, 2))
        return set_error(TTT_ERR_INVALID_ARG, "Out overlaps Q, K_new or V_new");
    if (q.ld_request == 0 && q.B > 1 && K_new) return set_error(TTT_ERR_INVALID_ARG, "the requests store into the same cache slots");
    if (K_new) {
        // a request's new key of one head must not land in another head's: heads lie within a slot or slots within a head
        const bool within_slot = (q.Hk - 1) * q.ld_head + q.d <= q.ld_slot && q.ld_head >= q.d;
        const bool within_head = (q.slots - 1) * q.ld_slot + q.d <= q.ld_head;
        if (q.Hk > 1 && !within_slot && !within_head)
            return set_error(TTT_ERR_INVALID_ARG, "ld_slot=%lld, ld_head=%lld: heads share cache slots", q.ld_slot, q.ld_head);
        if (K_cache == V_cache && K_new != V_new) return set_error(TTT_ERR_INVALID_ARG, "keys and values are stored into the same cache");
    }
    WindowDecodeArgs a{};
    a.B = q.B; a.Hq = q.Hq; a.Hk = q.Hk; a.slots = q.slots; a.left = q.left; a.sinks = q.sinks; a.scale = q.scale;
    a.ld_request = q.ld_request; a.ld_slot = q.ld_slot; a.ld_head = q.ld_head;
    a.Q = static_cast<const __nv_bfloat16*>(Q); a.ld_q = ld_q;
    a.K_new = static_cast<const __nv_bfloat16*>(K_new); a.V_new = static_cast<const __nv_bfloat16*>(V_new); a.ld_new = ld_new;
    a.K_cache = static_cast<__nv_bfloat16*>(K_cache); a.V_cache = static_cast<__nv_bfloat16*>(V_cache);
    a.lens = lens;
    a.Out = static_cast<__nv_bfloat16*>(Out); a.ld_out = ld_out;
    a.status = static_cast<int*>(workspace);
    SEQ_TRY(launch_window_decode(a, reinterpret_cast<cudaStream_t>(stream)));
    return TTT_OK;
}

// ---------------------------------------------------------------- gated linear recurrence
static ttt_status check_gated(const ttt_gated_scan_desc* q) {
    if (!q) return set_error(TTT_ERR_INVALID_ARG, "desc is NULL");
    if (q->T < 0 || q->T > kMaxRows) return set_error(TTT_ERR_INVALID_ARG, "T=%d must lie in [0, 2^30]", q->T);
    if (q->D < 8 || q->D % 8) return set_error(TTT_ERR_INVALID_ARG, "D=%d must be a positive multiple of 8", q->D);
    if (q->n_seq < 1 || q->n_seq > kMaxRows) return set_error(TTT_ERR_INVALID_ARG, "n_seq=%d must be at least 1", q->n_seq);
    if (q->form < TTT_GATE_SUM || q->form > TTT_GATE_UNIT) return set_error(TTT_ERR_INVALID_ARG, "form %d", (int)q->form);
    if (q->dir != TTT_FWD && q->dir != TTT_REV) return set_error(TTT_ERR_INVALID_ARG, "dir must be TTT_FWD or TTT_REV");
    if (q->x_dtype != TTT_F32 && q->x_dtype != TTT_BF16) return set_error(TTT_ERR_INVALID_ARG, "x_dtype %d", (int)q->x_dtype);
    return TTT_OK;
}

extern "C" TTT_API size_t ttt_gated_scan_workspace_size(const ttt_gated_scan_desc* desc) {
    if (check_gated(desc) != TTT_OK) return 0;
    return kAlign;
}

extern "C" TTT_API size_t ttt_gated_scan_chunk_states_size(const ttt_gated_scan_desc* desc) {
    if (check_gated(desc) != TTT_OK) return 0;
    return align_up((size_t)std::max(1LL, gated_scan_chunk_state_floats(desc->T, desc->D)) * sizeof(float));
}

static void fill_gated(GatedScanArgs& a, const ttt_gated_scan_desc& q, const int* cu, const void* F, int ld_f,
                       const void* X, int ld_x, const float* H_0, void* workspace) {
    a.T = q.T; a.D = q.D; a.n_seq = q.n_seq; a.form = (int)q.form; a.reverse = q.dir == TTT_REV;
    a.bf16 = q.x_dtype == TTT_BF16;
    a.cu = cu; a.F = F; a.ld_f = ld_f; a.X = X; a.ld_x = ld_x; a.H_0 = H_0;
    a.status = static_cast<int*>(workspace);
}

static ttt_status check_state(const void* p, const char* name) { return p ? need(p, name) : TTT_OK; }

extern "C" TTT_API ttt_status ttt_gated_scan(const ttt_gated_scan_desc* desc, const int* cu, const void* F, int ld_f,
                                     const void* X, int ld_x, const float* H_0, void* Y, int ld_y, float* H_T,
                                     void* chunk_states, void* workspace, size_t workspace_bytes,
                                     ttt_stream_t stream) {
    SEQ_NEED(check_gated(desc));
    const ttt_gated_scan_desc& q = *desc;
    SEQ_NEED(check_sequences(q.n_seq, cu));
    SEQ_NEED(check_workspace(workspace, workspace_bytes, ttt_gated_scan_workspace_size(desc)));
    if (q.T) {
        SEQ_NEED(need_rows(F, ld_f, q.D, "F"));
        SEQ_NEED(need_rows(X, ld_x, q.D, "X"));
        SEQ_NEED(need_rows(Y, ld_y, q.D, "Y"));
    }
    SEQ_NEED(check_state(H_0, "H_0"));
    SEQ_NEED(check_state(H_T, "H_T"));
    SEQ_NEED(check_state(chunk_states, "chunk_states"));
    const size_t e = q.x_dtype == TTT_BF16 ? 2 : 4;
    if (overlap(Y, q.T, ld_y, q.D, e, F, q.T, ld_f, q.D, e) || overlap(Y, q.T, ld_y, q.D, e, X, q.T, ld_x, q.D, e))
        return set_error(TTT_ERR_INVALID_ARG, "Y overlaps F or X");
    if (overlap(H_T, q.n_seq, q.D, q.D, 4, H_0, q.n_seq, q.D, q.D, 4))
        return set_error(TTT_ERR_INVALID_ARG, "H_T overlaps H_0");
    GatedScanArgs a{};
    fill_gated(a, q, cu, F, ld_f, X, ld_x, H_0, workspace);
    a.Y = Y; a.ld_y = ld_y; a.H_T = H_T; a.chunk_states = static_cast<float*>(chunk_states);
    SEQ_TRY(launch_gated_scan(a, reinterpret_cast<cudaStream_t>(stream)));
    return TTT_OK;
}

extern "C" TTT_API ttt_status ttt_gated_scan_backward(const ttt_gated_scan_desc* desc, const int* cu, const void* F, int ld_f,
                                              const void* X, int ld_x, const float* H_0, const void* chunk_states,
                                              const void* dY, int ld_dy, const float* dH_T, void* dF, int ld_df,
                                              void* dX, int ld_dx, float* dH_0, void* workspace,
                                              size_t workspace_bytes, ttt_stream_t stream) {
    SEQ_NEED(check_gated(desc));
    const ttt_gated_scan_desc& q = *desc;
    SEQ_NEED(check_sequences(q.n_seq, cu));
    SEQ_NEED(check_workspace(workspace, workspace_bytes, ttt_gated_scan_workspace_size(desc)));
    if (q.T) {
        SEQ_NEED(need_rows(F, ld_f, q.D, "F"));
        SEQ_NEED(need_rows(X, ld_x, q.D, "X"));
        SEQ_NEED(need_rows(dY, ld_dy, q.D, "dY"));
        SEQ_NEED(need_rows(dF, ld_df, q.D, "dF"));
        SEQ_NEED(need_rows(dX, ld_dx, q.D, "dX"));
        SEQ_NEED(need(chunk_states, "chunk_states"));
    }
    SEQ_NEED(check_state(H_0, "H_0"));
    SEQ_NEED(check_state(dH_T, "dH_T"));
    SEQ_NEED(check_state(dH_0, "dH_0"));
    const size_t e = q.x_dtype == TTT_BF16 ? 2 : 4;
    struct Rows { const void* p; long long ld; };
    const Rows in[] = {{F, ld_f}, {X, ld_x}, {dY, ld_dy}};
    const Rows out[] = {{dF, ld_df}, {dX, ld_dx}};
    for (const Rows& o : out)
        for (const Rows& r : in)
            if (overlap(o.p, q.T, o.ld, q.D, e, r.p, q.T, r.ld, q.D, e))
                return set_error(TTT_ERR_INVALID_ARG, "a gradient overlaps an input");
    if (overlap(dF, q.T, ld_df, q.D, e, dX, q.T, ld_dx, q.D, e)) return set_error(TTT_ERR_INVALID_ARG, "dF overlaps dX");
    if (overlap(dH_0, q.n_seq, q.D, q.D, 4, dH_T, q.n_seq, q.D, q.D, 4) ||
        overlap(dH_0, q.n_seq, q.D, q.D, 4, H_0, q.n_seq, q.D, q.D, 4))
        return set_error(TTT_ERR_INVALID_ARG, "dH_0 overlaps dH_T or H_0");
    GatedScanArgs a{};
    fill_gated(a, q, cu, F, ld_f, X, ld_x, H_0, workspace);
    a.chunk_states = static_cast<float*>(const_cast<void*>(chunk_states));
    a.dY = dY; a.ld_dy = ld_dy; a.dH_T = dH_T;
    a.dF = dF; a.ld_df = ld_df; a.dX = dX; a.ld_dx = ld_dx; a.dH_0 = dH_0;
    SEQ_TRY(launch_gated_scan_backward(a, reinterpret_cast<cudaStream_t>(stream)));
    return TTT_OK;
}

extern "C" TTT_API ttt_status ttt_gated_scan_step(int B, int D, ttt_gate_form form, ttt_dtype x_dtype, const void* F, int ld_f,
                                          const void* X, int ld_x, const float* H, float* H_out, void* Y, int ld_y,
                                          ttt_stream_t stream) {
    const ttt_gated_scan_desc q{B, D, 1, form, TTT_FWD, x_dtype};
    SEQ_NEED(check_gated(&q));
    if (B == 0) return TTT_OK;
    SEQ_NEED(need_rows(F, ld_f, D, "F"));
    SEQ_NEED(need_rows(X, ld_x, D, "X"));
    SEQ_NEED(need(H, "H"));
    SEQ_NEED(need(H_out, "H_out"));
    if (Y) SEQ_NEED(need_rows(Y, ld_y, D, "Y"));
    const size_t e = x_dtype == TTT_BF16 ? 2 : 4;
    if (H_out != H && overlap(H_out, B, D, D, 4, H, B, D, D, 4))
        return set_error(TTT_ERR_INVALID_ARG, "H_out overlaps H and is not H itself");
    if (Y && (overlap(Y, B, ld_y, D, e, F, B, ld_f, D, e) || overlap(Y, B, ld_y, D, e, X, B, ld_x, D, e)))
        return set_error(TTT_ERR_INVALID_ARG, "Y overlaps F or X");
    if (overlap(H_out, B, D, D, 4, F, B, ld_f, D, e) || overlap(H_out, B, D, D, 4, X, B, ld_x, D, e) ||
        overlap(Y, B, ld_y, D, e, H, B, D, D, 4) || overlap(Y, B, ld_y, D, e, H_out, B, D, D, 4))
        return set_error(TTT_ERR_INVALID_ARG, "H_out overlaps F or X, or Y overlaps a state");
    SEQ_TRY(launch_gated_scan_step(B, D, (int)form, x_dtype == TTT_BF16, F, ld_f, X, ld_x, H, H_out, Y, ld_y,
                                   reinterpret_cast<cudaStream_t>(stream)));
    return TTT_OK;
}
