// zsp_head.cpp -- entry points of the losses over the head (zsp_head_loss,
// zsp_head_distill, zsp_head_workspace): argument checks, the layout of the
// workspace, and how a call is cut.
#include <algorithm>
#include <cmath>

#include "zsp_entry.hpp"
#include "zsp_head.hpp"

namespace zsp {
namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 23, kMaxVocab = int64_t(1) << 22, kMaxDepth = 65536;
// The softmax of at most so many bytes is kept at a time, or of a tile's tokens
// where those take more (fp32 beyond 1.6 million columns; 10.7 GB at 2^22).
constexpr int64_t kKeptBytes = int64_t(1) << 32;

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// The workspace's parts, one behind another. All grow with the tokens but the
// copy of X^T, which calls of more than a few do without, and the parts of sums
// (split_bytes).
void lay_out(HeadShape* s) {
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = at;
        at = up(at + bytes, 256);
        return o;
    };
    const bool grads = s->grad_hidden || s->grad_head;
    s->o_count = take(4);
    s->o_rows = take(s->rows * 4);
    s->o_coef = take(s->rows * 4);
    s->o_entry = take(s->rows * s->top_pad * 4);
    s->o_pick = take(s->rows * s->top_pad * 4);
    if (s->teacher) {
        s->o_flag = take(s->n);
        s->o_teach = take(s->rows * s->top_pad * 4);
        if (s->top > 1) s->o_start = take(s->n * ((s->v + kHeadBlock - 1) / kHeadBlock + 1) * 2);
    }
    s->o_x = take(s->rows * s->dp * 2 * s->planes);
    s->o_xt = take(s->xt_tokens * s->dp * 2);
    if (s->pack_head) s->o_w = take(s->v * s->dp * 2 * s->planes);
    s->o_part = take(s->chunk * (s->vp / kHeadBlock) * 8);
    if (grads) s->o_p = take(s->chunk * s->vp * (s->f32 ? 4 : 2));
    if (grads && s->f32) s->o_g = take(s->chunk * s->vp * 2 * s->planes);
    s->o_split = take(s->split_bytes);
    if (s->grad_head && s->nchunk > 1) s->o_acc = take(s->v * s->dp * 4);
    s->bytes = at;
}

// What a call of n tokens takes.
zsp_status make_shape(int64_t n, int64_t v, int64_t d, zsp_dtype dtype, int32_t top,
                      int32_t flags, HeadShape* out) {
    if (dtype != ZSP_F32 && dtype != ZSP_BF16) return set_error(ZSP_EINVAL, "bad dtype %d", dtype);
    if (n < 0 || v < 1 || d < 1 || top < 0)
        return set_error(ZSP_EINVAL, "n = %lld, v = %lld, d = %lld, top = %d", (long long)n,
                         (long long)v, (long long)d, top);
    if (flags & ~(ZSP_HEAD_GRAD_HIDDEN | ZSP_HEAD_GRAD_HEAD | ZSP_HEAD_UNALIGNED))
        return set_error(ZSP_EINVAL, "bad flags %d", flags);
    if (n > kMaxTokens || v > kMaxVocab || d > kMaxDepth || top > kHeadMaxTop)
        return set_error(ZSP_ERANGE, "n = %lld, v = %lld, d = %lld or top = %d is too large",
                         (long long)n, (long long)v, (long long)d, top);
    HeadShape s;
    s.n = n;
    s.v = v;
    s.d = d;
    s.f32 = dtype == ZSP_F32;
    s.teacher = top > 0;
    s.top = std::max(top, 1);
    s.top_pad = s.top == 1 ? 1 : int32_t(up(s.top, 4));
    s.grad_hidden = flags & ZSP_HEAD_GRAD_HIDDEN;
    s.grad_head = flags & ZSP_HEAD_GRAD_HEAD;
    s.planes = s.f32 ? 3 : 1;
    // up to 64 tokens are in tiles of at most 64: one of 2^22 fp32 columns would
    // else keep 10.7 GB, and keeps 2.7
    const int64_t tile = n <= kHeadThin ? kHeadThin : kHeadTile;
    s.rows = up(n, tile);
    s.vp = up(v, kHeadTile);
    s.dp = up(d, kHeadDepth);
    const bool aligned = !(flags & ZSP_HEAD_UNALIGNED);
    s.in_place = s.f32 && d % 4 == 0 && aligned;
    s.thin = s.in_place && n <= kHeadThin;
    s.pack_head = s.f32 ? !s.thin : d % 8 != 0 || !aligned;
    if (s.grad_head && !s.f32 && n <= kHeadFew) s.xt_tokens = up(n, 32);
    const bool grads = s.grad_hidden || s.grad_head;
    // per token: P (and its planes), or the partials alone
    const int64_t per = grads ? s.vp * (s.f32 ? 4 + 2 * s.planes : 2) : s.vp / kHeadBlock * 8;
    s.chunk_most = std::max<int64_t>(kKeptBytes / per / kHeadTile * kHeadTile, kHeadTile);
    s.nchunk = std::max<int64_t>((n + s.chunk_most - 1) / s.chunk_most, 1);
    s.chunk = up((n + s.nchunk - 1) / s.nchunk, tile);
    if (s.chunk > 0) s.nchunk = std::max<int64_t>((n + s.chunk - 1) / s.chunk, 1);
    if (!head_fits_launch(s))
        return set_error(ZSP_ERANGE, "n * d = %lld * %lld elements are too many", (long long)n,
                         (long long)d);
    head_products(&s);
    lay_out(&s);
    *out = s;
    return ZSP_OK;
}

struct Span {
    const char* what;
    const void* p;
    int64_t bytes;
    int32_t align;
    bool written;
};

// Pointers present and aligned, and nothing written that another argument holds.
zsp_status check_spans(const Span* s, int n) {
    for (int i = 0; i < n; ++i) {
        if (!s[i].p || s[i].bytes == 0) continue;
        if (reinterpret_cast<uintptr_t>(s[i].p) % uintptr_t(s[i].align))
            return set_error(ZSP_EINVAL, "%s is not aligned to %d bytes", s[i].what, s[i].align);
    }
    for (int i = 0; i < n; ++i) {
        if (!s[i].written || !s[i].p || s[i].bytes == 0) continue;
        const uintptr_t a = reinterpret_cast<uintptr_t>(s[i].p), ae = a + uintptr_t(s[i].bytes);
        for (int j = 0; j < n; ++j) {
            if (j == i || !s[j].p || s[j].bytes == 0) continue;
            const uintptr_t b = reinterpret_cast<uintptr_t>(s[j].p);
            if (a < b + uintptr_t(s[j].bytes) && b < ae)
                return set_error(ZSP_EINVAL, "%s overlaps %s", s[i].what, s[j].what);
        }
    }
    return ZSP_OK;
}

zsp_status head_call(HeadCall c, int64_t n, int64_t v, int64_t d, zsp_dtype dtype, int32_t top,
                     int64_t ws_bytes, void* stream) {
    int32_t flags = (c.grad_hidden ? ZSP_HEAD_GRAD_HIDDEN : 0) |
                    (c.grad_head ? ZSP_HEAD_GRAD_HEAD : 0) |
                    (reinterpret_cast<uintptr_t>(c.head) % 16 ? ZSP_HEAD_UNALIGNED : 0);
    HeadShape s;
    zsp_status st = make_shape(n, v, d, dtype, top, flags, &s);
    if (st != ZSP_OK) return st;
    // the softmax's exponents are taken in units of T / log2(e)
    if (!(c.temperature > 0.0f) || !std::isfinite(c.temperature) ||
        !std::isfinite(1.0f / c.temperature * 1.4426950408889634f))
        return set_error(ZSP_EINVAL,
                         "temperature = %g is not above 0, or 1.4427 times its inverse not finite",
                         double(c.temperature));
    if (!std::isfinite(c.scale) || !std::isfinite(c.scale * c.temperature))
        return set_error(ZSP_EINVAL, "scale is not finite, or its product with the temperature");
    if (!c.head) return set_error(ZSP_EINVAL, "head is NULL");
    if (!c.ws) return set_error(ZSP_EINVAL, "ws is NULL");
    if (n > 0) {
        if (!c.hidden) return set_error(ZSP_EINVAL, "hidden is NULL");
        if (!c.index) return set_error(ZSP_EINVAL, top ? "index is NULL" : "target is NULL");
        if (top && !c.logit) return set_error(ZSP_EINVAL, "logit is NULL");
        if (!c.loss) return set_error(ZSP_EINVAL, "loss is NULL");
    }
    const int32_t e = s.f32 ? 4 : 2;
    const Span spans[] = {
        {"hidden", c.hidden, n * d * e, e, false},
        {"head", c.head, v * d * e, e, false},
        {top ? "index" : "target", c.index, n * s.top * 8, 8, false},
        {"logit", c.logit, n * s.top * 4, 4, false},
        {"token_weight", c.token_weight, n * 4, 4, false},
        {"loss", c.loss, n * 4, 4, true},
        {"lse", c.lse, n * 4, 4, true},
        {"grad_hidden", c.grad_hidden, n * d * e, e, true},
        {"grad_head", c.grad_head, v * d * e, e, true},
        {"ws", c.ws, ws_bytes, 16, true},
    };
    if (ws_bytes < s.bytes)
        return set_error(ZSP_ERANGE, "ws_bytes = %lld, %lld are needed", (long long)ws_bytes,
                         (long long)s.bytes);
    if ((st = check_spans(spans, int(sizeof(spans) / sizeof(spans[0])))) != ZSP_OK) return st;
    const hipError_t err = launch_head(s, c, static_cast<hipStream_t>(stream));
    if (err != hipSuccess) return set_hip_error(err, "head loss launch");
    return ZSP_OK;
}

}  // namespace
}  // namespace zsp

extern "C" {

zsp_status zsp_head_workspace(int64_t n, int64_t v, int64_t d, zsp_dtype dtype, int32_t top,
                              int32_t flags, int64_t* bytes) {
    using namespace zsp;
    if (!bytes) return set_error(ZSP_EINVAL, "bytes is NULL");
    // the most of the calls with some of the gradients, which may keep more
    // tokens at a time, and with up to n tokens, whose parts of sums or chunks may
    // be larger
    const int32_t grads = flags & (ZSP_HEAD_GRAD_HIDDEN | ZSP_HEAD_GRAD_HEAD);
    int64_t most = 0;
    for (int32_t some = 0; some <= grads; ++some) {
        if (some & ~grads) continue;
        HeadShape s;
        const zsp_status st = make_shape(n, v, d, dtype, top, (flags & ~grads) | some, &s);
        if (st != ZSP_OK) return st;
        s.split_bytes = head_split_most(s);
        s.chunk = std::min(s.rows, s.chunk_most);
        if (s.grad_head && !s.f32) s.xt_tokens = up(std::min<int64_t>(n, kHeadFew), 32);
        lay_out(&s);
        most = std::max(most, s.bytes);
    }
    *bytes = most;
    return ZSP_OK;
}

zsp_status zsp_head_loss(const void* hidden, const void* head, zsp_dtype dtype, int64_t n,
                         int64_t v, int64_t d, const int64_t* target, const float* token_weight,
                         float scale, float* loss, float* lse, void* grad_hidden, void* grad_head,
                         void* ws, int64_t ws_bytes, void* stream) {
    using namespace zsp;
    const HeadCall c{hidden, head, target, nullptr, token_weight, scale, 1.0f, loss, lse,
                     grad_hidden, grad_head, static_cast<char*>(ws)};
    return head_call(c, n, v, d, dtype, 0, ws_bytes, stream);
}

zsp_status zsp_head_distill(const void* hidden, const void* head, zsp_dtype dtype, int64_t n,
                            int64_t v, int64_t d, const int64_t* index, const float* logit,
                            int32_t top, float temperature, const float* token_weight, float scale,
                            float* loss, float* lse, void* grad_hidden, void* grad_head, void* ws,
                            int64_t ws_bytes, void* stream) {
    using namespace zsp;
    if (top < 1) return set_error(ZSP_EINVAL, "top = %d is below 1", top);
    const HeadCall c{hidden, head, index, logit, token_weight, scale, temperature, loss, lse,
                     grad_hidden, grad_head, static_cast<char*>(ws)};
    return head_call(c, n, v, d, dtype, top, ws_bytes, stream);
}

}  // extern "C"
