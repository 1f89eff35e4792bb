// C ABI of the cache append, the tree attention and the logit penalties
// (declared in include/w4a8.h): argument checks and launch plans.  No entry
// point allocates memory or synchronises.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/w4a8.h"
#include "attention.h"

using namespace w4k;

static_assert(W4_I8 == T_I8, "public element types");
static_assert(W4_MAX_SEQUENCES == kAtMaxSeq && W4_MAX_DRAFTS == kAtMaxTok && W4_MAX_BIASES == kLgMaxBias, "public limits");

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline w4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? W4_OK : W4_ERR_CUDA; }
inline bool elem_type(int t) { return t == W4_F32 || t == W4_F16 || t == W4_BF16; }
inline bool half_type(int t) { return t == W4_F16 || t == W4_BF16; }

constexpr int kMaxHeads = 1024;
constexpr long long kMaxPlaces = 1ll << 30;
constexpr int kMaxHistory = 1 << 28;                      // (tokens are counted in fours and walked in 32 bits)
constexpr long long kMaxUnits = 0x7fffffffll - 1024;      // (the kernels count units of work in 32 bits)

int log2_of(int v)
{
    int n = 0;
    while ((1 << n) < v) ++n;
    return n;
}

w4_status check_cache(const w4_kv_cache* c)
{
    if (!c) return W4_ERR_INVALID_ARG;
    if ((!half_type(c->type) && c->type != W4_I8) || c->pages < 1 || c->page_size < 1 || c->Hkv < 1 || c->D < 1)
        return W4_ERR_INVALID_ARG;
    if (c->D != 64 && c->D != 128 && c->D != 256) return W4_ERR_UNSUPPORTED_SHAPE;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0) return W4_ERR_UNSUPPORTED_SHAPE;
    return static_cast<long long>(c->pages) * c->Hkv > 0x7fffffffll ? W4_ERR_UNSUPPORTED_SHAPE : W4_OK;
}

// Numbers of a call on a cache; its pointers come after the empty calls.
w4_status check_call(const w4_kv_cache* c, const w4_kv_batch* b, int T, int Hq)
{
    if (!b || T < 0 || Hq <= 0 || b->B < 0 || b->max_pages < 1 || b->max_tokens < 1) return W4_ERR_INVALID_ARG;
    const w4_status r = check_cache(c);
    if (r != W4_OK) return r;
    if (Hq % c->Hkv != 0 || Hq > kMaxHeads || T > W4_MAX_TOKENS || b->B > W4_MAX_SEQUENCES) return W4_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<long long>(b->max_pages) * c->page_size > kMaxPlaces)
        return W4_ERR_UNSUPPORTED_SHAPE;
    return W4_OK;
}

w4_status check_cache_pointers(const w4_kv_cache* c)
{
    const bool i8 = c->type == W4_I8;
    if (!c->k || !c->v || i8 != (c->k_scale != nullptr) || i8 != (c->v_scale != nullptr)) return W4_ERR_INVALID_ARG;
    return aligned(c->k, 16) && aligned(c->v, 16) && aligned(c->k_scale, 16) && aligned(c->v_scale, 16) ? W4_OK : W4_ERR_MISALIGNED;
}
w4_status check_call_pointers(const w4_kv_cache* c, const w4_kv_batch* b)
{
    const w4_status r = check_cache_pointers(c);
    if (r == W4_ERR_INVALID_ARG || !b->table || !b->ctx || !b->q_start) return W4_ERR_INVALID_ARG;
    if (r != W4_OK || !aligned(b->table, 4) || !aligned(b->ctx, 4) || !aligned(b->q_start, 4))
        return W4_ERR_MISALIGNED;
    return W4_OK;
}

KvView view(const w4_kv_cache* c)
{
    return KvView{c->k, c->v, c->k_scale, c->v_scale, c->type, c->pages, c->page_size, log2_of(c->page_size), c->Hkv, c->D};
}
BatchView view(const w4_kv_batch* b) { return BatchView{b->table, b->ctx, b->q_start, b->B, b->max_pages, b->max_tokens}; }

// Which kernel a call takes, and the rows of its partial results.  Up to 16 rows to a key head are one tile of the mma.sync
// kernel; more would read the cache again for every 16, where the tcgen05 kernel takes 128.  28 query and 4 key heads of 128,
// 3 drafts (21 rows): 65536 bf16 places 42 us on tcgen05, 45.6 on mma.sync; INT8 50 and 55.6; 30 streams of 400 to 4000
// places 36.7 and 48.2; 4096 places 12.0 and 11.3.  8 query heads of 256 over one key head, 3 drafts (24 rows), 120001 INT8 places:
// 42.8 and 65.2.
struct AttnPlan {
    bool tc;
    int part_rows;
    long long units;          // of work, at most
};
AttnPlan plan_attention(const w4_kv_cache* c, const w4_kv_batch* b, int T, int G)
{
    const int rows = (b->max_tokens < T ? b->max_tokens : T) * G;
    AttnPlan p;
    p.tc = rows > kAtRows;
    const int tile = p.tc ? kAtTcRows : kAtRows, unit = p.tc ? kAtTcUnit : kAtUnit;
    p.units = static_cast<long long>(b->B) * c->Hkv * ((rows + tile - 1) / tile) *
              ((static_cast<long long>(b->max_pages) * c->page_size + unit - 1) / unit);
    p.part_rows = rows < tile ? (rows + 7) / 8 * 8 : tile;   // (results begin on 16-byte boundaries)
    return p;
}
size_t attention_workspace(const w4_kv_cache* c, const w4_kv_batch* b, const AttnPlan& p)
{
    const size_t block = 2 * attn_part_floats(p.part_rows, c->D) + (p.tc ? static_cast<size_t>(p.part_rows) * c->D : 0);
    return attn_head_bytes(b->B) + kAtMaxBlocks * block * 4;
}

}  // namespace

extern "C" {

w4_status w4_rope_table(const double* inv_freq, double factor, double scale, int positions, int rot, float* turns,
                        w4_stream_t s)
{
    if (positions < 0 || rot < 0 || !(factor > 0.0) || !(scale > 0.0)) return W4_ERR_INVALID_ARG;
    if (rot % 8 != 0 || rot > 256 || positions > (1 << 26)) return W4_ERR_UNSUPPORTED_SHAPE;
    if (positions == 0 || rot == 0) return W4_OK;
    if (!inv_freq || !turns) return W4_ERR_INVALID_ARG;
    if (!aligned(inv_freq, 8) || !aligned(turns, 16)) return W4_ERR_MISALIGNED;
    return cuda_status(launch_rope_table(inv_freq, factor, scale, positions, rot / 2, turns, reinterpret_cast<cudaStream_t>(s)));
}

w4_status w4_kv_append(const w4_kv_cache* c, const w4_kv_batch* b, const w4_rope* rope, const void* qkv, int x_type,
                       long long ld, int T, int Hq, const int* positions, const float* q_norm, const float* k_norm,
                       float eps, void* q, int q_type, unsigned flags, w4_stream_t s)
{
    w4_status r = check_call(c, b, T, Hq);
    if (r != W4_OK) return r;
    if (!elem_type(x_type) || !half_type(q_type) || (flags & ~W4_FLAG_PDL) != 0) return W4_ERR_INVALID_ARG;
    const long long width = static_cast<long long>(Hq + 2 * c->Hkv) * c->D;
    if (ld < width) return W4_ERR_INVALID_ARG;
    if ((q_norm || k_norm) && (!(eps > 0.0f) || !(eps < 3.0e38f))) return W4_ERR_INVALID_ARG;
    if (rope && (rope->rot < 0 || rope->positions < 1 || (rope->layout != W4_ROPE_HALF && rope->layout != W4_ROPE_INTERLEAVED)))
        return W4_ERR_INVALID_ARG;
    if (rope && (rope->rot % 8 != 0 || rope->rot > c->D)) return W4_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || b->B == 0) return W4_OK;
    r = check_call_pointers(c, b);
    if (r == W4_ERR_INVALID_ARG || !qkv || !q || (rope && rope->rot > 0 && !rope->turns)) return W4_ERR_INVALID_ARG;
    if (r != W4_OK || !aligned(qkv, 16) || ld * elem_bytes(x_type) % 16 != 0 || !aligned(q, 16) || !aligned(positions, 4) ||
        !aligned(q_norm, 16) || !aligned(k_norm, 16) || (rope && !aligned(rope->turns, 16)))
        return W4_ERR_MISALIGNED;
    AppendArgs a = {};
    a.c = view(c);
    a.b = view(b);
    a.x = qkv;
    a.ld = ld;
    a.T = T;
    a.Hq = Hq;
    if (rope) {
        a.turns = rope->turns;
        a.positions = rope->positions;
        a.rot = rope->rot;
        a.interleaved = rope->layout == W4_ROPE_INTERLEAVED;
    }
    a.pos = positions;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.eps = eps;
    a.q = q;
    a.qtype = q_type;
    return cuda_status(launch_kv_append(a, x_type, reinterpret_cast<cudaStream_t>(s)));
}

w4_status w4_kv_values(const w4_kv_cache* c, int which, float* out, w4_stream_t s)
{
    w4_status r = check_cache(c);
    if (r != W4_OK) return r;
    if (c->type != W4_I8 || (which != W4_KEYS && which != W4_VALUES)) return W4_ERR_INVALID_ARG;
    if (static_cast<long long>(c->pages) * c->Hkv * c->page_size * (c->D / 8) > (1ll << 38)) return W4_ERR_UNSUPPORTED_SHAPE;
    r = check_cache_pointers(c);
    if (r == W4_ERR_INVALID_ARG || !out) return W4_ERR_INVALID_ARG;
    if (r != W4_OK || !aligned(out, 16)) return W4_ERR_MISALIGNED;
    return cuda_status(launch_kv_values(view(c), which == W4_VALUES, out, reinterpret_cast<cudaStream_t>(s)));
}

size_t w4_tree_attention_workspace_bytes(const w4_kv_cache* c, const w4_kv_batch* b, int T, int Hq)
{
    if (check_call(c, b, T, Hq) != W4_OK || b->max_tokens > W4_MAX_DRAFTS || T == 0 || b->B == 0) return 0;
    const AttnPlan p = plan_attention(c, b, T, Hq / c->Hkv);
    return p.units <= kMaxUnits ? attention_workspace(c, b, p) : 0;
}

w4_status w4_tree_attention(const w4_kv_cache* c, const w4_kv_batch* b, const void* q, int q_type, int T, int Hq,
                            const unsigned long long* mask, float scale, void* y, int y_type, void* workspace,
                            size_t ws_bytes, unsigned flags, w4_stream_t s)
{
    w4_status r = check_call(c, b, T, Hq);
    if (r != W4_OK) return r;
    if (!half_type(q_type) || (c->type != W4_I8 && q_type != c->type) || !elem_type(y_type) || (flags & ~W4_FLAG_PDL) != 0 ||
        !(scale > 0.0f) || !(scale < 2.0e38f))             // (times log2(e) it is an fp32 number)
        return W4_ERR_INVALID_ARG;
    if (b->max_tokens > W4_MAX_DRAFTS) return W4_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || b->B == 0) return W4_OK;
    r = check_call_pointers(c, b);
    if (r == W4_ERR_INVALID_ARG || !q || !y || !workspace) return W4_ERR_INVALID_ARG;
    const AttnPlan p = plan_attention(c, b, T, Hq / c->Hkv);
    if (p.units > kMaxUnits || ws_bytes < attention_workspace(c, b, p)) return W4_ERR_UNSUPPORTED_SHAPE;
    if (r != W4_OK || !aligned(q, 16) || !aligned(y, 16) || !aligned(mask, 8) || !aligned(workspace, 16)) return W4_ERR_MISALIGNED;
    DeviceFacts d;
    if (!device_facts(&d)) return W4_ERR_CUDA;
    AttnArgs a = {};
    a.c = view(c);
    a.b = view(b);
    a.q = q;
    a.mask = mask;
    a.scale = scale * 1.4426950408889634f;
    a.T = T;
    a.Hq = Hq;
    a.G = Hq / c->Hkv;
    a.y = y;
    a.ytype = y_type;
    a.head = static_cast<int*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + attn_head_bytes(b->B));
    a.part_rows = p.part_rows;
    a.units = p.units;
    a.kept = a.part + kAtMaxBlocks * 2 * attn_part_floats(p.part_rows, c->D);
    a.err = d.err;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
    const cudaError_t e = p.tc ? launch_attn_tc(a, q_type, d.sms, cs) : launch_attn_tree(a, q_type, d.sms, cs);
    if (e != cudaSuccess) return W4_ERR_CUDA;
    return cuda_status(p.tc ? launch_attn_join(a, kAtTcRows, kAtTcUnit, cs) : launch_attn_join(a, kAtRows, kAtUnit, cs));
}

w4_status w4_logits_adjust(const w4_logit_rules* u, const void* logits, int type, long long ld, int R, const int* row_start,
                           const int* drafts, const unsigned long long* mask, const unsigned* allowed, void* out,
                           long long ld_out, unsigned flags, w4_stream_t s)
{
    if (!u || R < 0 || u->V < 0 || u->S < 0 || u->cap < 0 || u->n_bias < 0 || !elem_type(type) || (flags & ~W4_FLAG_PDL) != 0)
        return W4_ERR_INVALID_ARG;
    if (ld < u->V || ld_out < u->V || (drafts && !row_start) || (mask && !drafts) ||
        (logits == out && ld != ld_out && R > 1))
        return W4_ERR_INVALID_ARG;
    if (R > W4_MAX_TOKENS || u->V > (1 << 24) || static_cast<long long>(R) * u->V > (1ll << 42) || u->n_bias > W4_MAX_BIASES ||
        u->S > W4_MAX_TOKENS || u->cap > kMaxHistory)
        return W4_ERR_UNSUPPORTED_SHAPE;
    if (R == 0 || u->V == 0 || u->S == 0) return W4_OK;
    const bool hist = u->cap > 0, bias = u->n_bias > 0;
    if (!logits || !out || (hist && (!u->ids || !u->length)) || (bias && (!u->bias_ids || !u->bias))) return W4_ERR_INVALID_ARG;
    const size_t eb = static_cast<size_t>(elem_bytes(type));
    if (!aligned(logits, eb) || !aligned(out, eb) || !aligned(u->ids, 4) || !aligned(u->length, 4) || !aligned(u->prompt, 4) ||
        !aligned(u->repetition, 4) || !aligned(u->frequency, 4) || !aligned(u->presence, 4) || !aligned(u->bias_ids, 4) ||
        !aligned(u->bias, 4) || !aligned(row_start, 4) || !aligned(drafts, 4) || !aligned(mask, 8) || !aligned(allowed, 4))
        return W4_ERR_MISALIGNED;
    LogitArgs a = {};
    a.x = logits;
    a.y = out;
    a.ld = ld;
    a.ldy = ld_out;
    a.R = R;
    a.V = u->V;
    a.S = u->S;
    a.ids = hist ? u->ids : nullptr;
    a.length = u->length;
    a.prompt = u->prompt;
    a.cap = u->cap;
    a.rep = u->repetition;
    a.freq = u->frequency;
    a.pres = u->presence;
    a.bias_ids = bias ? u->bias_ids : nullptr;
    a.bias = u->bias;
    a.nb = u->n_bias;
    a.row_start = row_start;
    a.drafts = drafts;
    a.mask = mask;
    a.allowed = allowed;
    const size_t between = (reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(logits)) % 16;
    a.vec = between == 0 && (R == 1 || ((ld - ld_out) * static_cast<long long>(eb)) % 16 == 0);
    return cuda_status(launch_logits(a, type, reinterpret_cast<cudaStream_t>(s)));
}

}  // extern "C"
